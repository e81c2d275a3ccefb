// rotate_kernels.hip - norms of query and key heads and the position rotation
// in one pass, for gfx950.
//
// Each head vector is read once and written once (4 d bytes), which is all
// that bounds a prompt; a decoding step is a single short launch. The
// angles of a token serve all of its query and key heads, so a workgroup
// takes whole tokens: first one thread per (token, pair) forms the angle
// positions * inv_freq in binary64 and reduces it there to a turn in
// [-1/2, 1/2] (binary32 loses the angle of far positions: at 10^6 its step
// is 0.06), takes cos and sin of it in binary32 and leaves them in LDS; then
// d / 16 lanes take a vector, 8 pairs each, as two 16-byte chunks. A thread
// always holds the same chunk of its vectors, so the weights stay in
// registers.
#include "attend.h"
#include "kernels_common.h"

namespace kvc {
namespace {

struct RotateParams {
    RowsDev q_in, k_in, q_out, k_out;
    const uint16_t *q_weight, *k_weight;
    const int64_t* positions;
    uint32_t n, Hq, heads;  // heads: query and key heads of a token
    uint32_t n_pairs, pairing;
    float eps;
    float f[kMaxPairs];
};

__device__ __forceinline__ void unpack8(const kvc_u32x4& x, float (&y)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[2 * i] = bf16_lo(w[i]);
        y[2 * i + 1] = bf16_hi(w[i]);
    }
}

__device__ __forceinline__ kvc_u32x4 pack8(const float (&y)[8]) {
    return kvc_u32x4{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7])};
}

// Rows of queries and keys, of which each lane chooses. Kept in scalar registers:
// the compiler would turn the choice of a value into that of its address among the
// kernel's arguments, and read it from there for every vector (8191 tokens: 32.9 us,
// so 30.1).
struct Rows {
    uint64_t q, k, qts, kts, qhs, khs;  // addresses; strides in elements
};
__device__ __forceinline__ Rows rows_of(const RowsDev& q, const RowsDev& k) {
    Rows x{(uint64_t)q.data, (uint64_t)k.data, q.ts, k.ts, q.hs, k.hs};
    asm("" : "+s"(x.q), "+s"(x.k), "+s"(x.qts), "+s"(x.kts), "+s"(x.qhs), "+s"(x.khs));
    return x;
}
typedef __attribute__((address_space(1))) kvc_u32x4 global_u32x4;

// sum over the LPV (4 or 8) lanes of a vector
template <int LPV>
__device__ __forceinline__ float sum_lanes(float v) {
    v += dpp_xor1(v);
    v += dpp_xor2(v);
    if (LPV == 8)  // row_half_mirror: the other four lanes of eight
        v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x141, 0xF, 0xF, true));
    return v;
}

// TW tokens of one workgroup. Five waves a SIMD (a prompt of 8191 tokens: 30.1 us,
// with four 30.2; six spill: 39).
template <int D, int TW>
__global__ __launch_bounds__(kBlockThreads, 5) void norm_rotate_kernel(RotateParams p) {
    constexpr uint32_t LPV = D / 16;
    constexpr uint32_t VPB = kBlockThreads / LPV;  // vectors at a time
    __shared__ float cs[TW][kMaxPairs], sn[TW][kMaxPairs];
    const uint32_t tok0 = blockIdx.x * TW;
    const uint32_t ntok = p.n - tok0 < TW ? p.n - tok0 : TW;
    const uint32_t i = threadIdx.x % LPV;
    const uint32_t nrot = p.n_pairs / 8;  // lanes of a vector that hold pairs
    const bool turned = i < nrot;
    const uint32_t oa = turned && p.pairing == 0 ? 8 * i : 16 * i;
    const uint32_t ob = turned && p.pairing == 0 ? p.n_pairs + 8 * i : 16 * i + 8;
    // weights stay packed: registers bound how many vectors are on their way
    kvc_u32x4 wq[2] = {}, wk[2] = {};
    if (p.q_weight) {
        wq[0] = *reinterpret_cast<const kvc_u32x4*>(p.q_weight + oa);
        wq[1] = *reinterpret_cast<const kvc_u32x4*>(p.q_weight + ob);
    }
    if (p.k_weight) {
        wk[0] = *reinterpret_cast<const kvc_u32x4*>(p.k_weight + oa);
        wk[1] = *reinterpret_cast<const kvc_u32x4*>(p.k_weight + ob);
    }
    // the first vector's loads go out before the angles are taken, the next
    // one's before each is turned
    uint32_t t = 0, h = threadIdx.x / LPV;
    const auto settle = [&]() {
        while (h >= p.heads && t < ntok) {
            h -= p.heads;
            ++t;
        }
    };
    // the vector's row, from fields in registers
    const Rows in = rows_of(p.q_in, p.k_in), out = rows_of(p.q_out, p.k_out);
    const auto row_at = [&](const Rows& x) {
        const bool is_q = h < p.Hq;
        const uint64_t at = (tok0 + t) * (is_q ? x.qts : x.kts) + (is_q ? h : h - p.Hq) * (is_q ? x.qhs : x.khs);
        return (is_q ? x.q : x.k) + 2 * at;
    };
    kvc_u32x4 xa, xb;
    const auto load = [&]() {
        if (t >= ntok) return;
        const uint64_t x = row_at(in);
        xa = *(const global_u32x4*)(x + 2 * oa);
        xb = *(const global_u32x4*)(x + 2 * ob);
    };
    settle();
    load();
    for (uint32_t j = threadIdx.x; j < TW * kMaxPairs; j += kBlockThreads) {
        const uint32_t jt = j / kMaxPairs, pair = j % kMaxPairs;
        if (jt < ntok && pair < p.n_pairs) {
            const double turns = (double)p.positions[tok0 + jt] * (double)p.f[pair] * 0.15915494309189533577;
            const float r = 2.0f * (float)(turns - rint(turns));
            float s, c;
            sincospif(r, &s, &c);
            cs[jt][pair] = c;
            sn[jt][pair] = s;
        }
    }
    __syncthreads();
    while (t < ntok) {
        const bool is_q = h < p.Hq;
        const uint64_t y = row_at(out);
        global_u32x4 *const ya = (global_u32x4*)(y + 2 * oa), *const yb = (global_u32x4*)(y + 2 * ob);
        float a[8], b[8];
        unpack8(xa, a);
        unpack8(xb, b);
        const uint32_t t_now = t;
        h += VPB;
        settle();
        load();
        if (is_q ? p.q_weight != nullptr : p.k_weight != nullptr) {
            float ss = 0.0f;
#pragma unroll
            for (int u = 0; u < 8; ++u) ss = fmaf(a[u], a[u], fmaf(b[u], b[u], ss));
            ss = sum_lanes<LPV>(ss);
            const float inv = 1.0f / sqrtf(ss * (1.0f / D) + p.eps);
            float w[8];
            unpack8(is_q ? wq[0] : wk[0], w);
#pragma unroll
            for (int u = 0; u < 8; ++u) a[u] = a[u] * inv * w[u];
            unpack8(is_q ? wq[1] : wk[1], w);
#pragma unroll
            for (int u = 0; u < 8; ++u) b[u] = b[u] * inv * w[u];
        }
        if (turned) {
            float c[8], s[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                c[u] = cs[t_now][8 * i + u];
                s[u] = sn[t_now][8 * i + u];
            }
            if (p.pairing == 0) {
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float ra = fmaf(a[u], c[u], -(b[u] * s[u])), rb = fmaf(a[u], s[u], b[u] * c[u]);
                    a[u] = ra;
                    b[u] = rb;
                }
            } else {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float ra = fmaf(a[2 * u], c[u], -(a[2 * u + 1] * s[u]));
                    const float rb = fmaf(a[2 * u], s[u], a[2 * u + 1] * c[u]);
                    a[2 * u] = ra;
                    a[2 * u + 1] = rb;
                    const float rc = fmaf(b[2 * u], c[4 + u], -(b[2 * u + 1] * s[4 + u]));
                    const float rd = fmaf(b[2 * u], s[4 + u], b[2 * u + 1] * c[4 + u]);
                    b[2 * u] = rc;
                    b[2 * u + 1] = rd;
                }
            }
        }
        if (TW > 1) {  // a prompt's rows: 33.7 us with the hint, 35.1 without
            __builtin_nontemporal_store(pack8(a), ya);
            __builtin_nontemporal_store(pack8(b), yb);
        } else {
            *ya = pack8(a);
            *yb = pack8(b);
        }
    }
}

}  // namespace

hipError_t launch_norm_rotate(const RotateArgs& a, hipStream_t stream) {
    RotateParams p{};
    p.q_in = a.q_in;
    p.k_in = a.k_in;
    p.q_out = a.q_out;
    p.k_out = a.k_out;
    p.q_weight = static_cast<const uint16_t*>(a.q_weight);
    p.k_weight = static_cast<const uint16_t*>(a.k_weight);
    p.positions = a.positions;
    p.n = a.n;
    p.Hq = a.Hq;
    p.heads = a.Hq + a.Hk;
    p.n_pairs = a.n_pairs;
    p.pairing = a.pairing;
    p.eps = a.eps;
    for (uint32_t j = 0; j < a.n_pairs; ++j) p.f[j] = a.inv_freq[j];
    // From 4096 tokens on a workgroup takes four (every thread an angle) and stores past the caches, below one,
    // with plain stores. Calls over rows that no cache holds, 40 heads of 128, us, for one token a workgroup, one
    // with the hint, and two and four with it: 256 tokens 4.6, 4.2, 5.0, 6.6; 1024 7.3, 6.9, 7.7, 8.3; 2048 11.9,
    // 10.6, 10.3, 11.3; 4095 20.0, 19.3, 19.0, 18.8; 8191 33.4, 31.7, 32.3, 33.7 (5.0 TB/s). Not taken yet:
    // the hint with fewer tokens, 5 % from 256 tokens on.
    if (a.n >= 4096)
        return launch_kernel(a.d == 64 ? norm_rotate_kernel<64, 4> : norm_rotate_kernel<128, 4>, dim3((a.n + 3) / 4),
                             dim3(kBlockThreads), stream, p);
    return launch_kernel(a.d == 64 ? norm_rotate_kernel<64, 1> : norm_rotate_kernel<128, 1>, dim3(a.n),
                         dim3(kBlockThreads), stream, p);
}

}  // namespace kvc
