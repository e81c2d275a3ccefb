// attend_kernels.hip - attention of one new token over a paged cache or one
// layer of the shared pool, for gfx950.
//
// For one kv head, the query heads that share it (of one sequence, or of all
// agents of a pool) are the rows of a small matrix Q. A wave walks the tokens
// in tiles of 32 with one pass over the data (running maximum m and sum l):
//     S^T = K Q^T          16x16x32 matrix instructions, tokens x rows
//     p = exp2(S - m)      in the lanes that hold S
//     O^T += V^T p^T       16x16x32, channels x rows
// Operand order makes every exchange between lanes fall away: in both products
// a lane's column is one query row (lane % 16), so m, l and the rescaling are
// its own registers; and S^T leaves lane (g, c) with tokens 4g..4g+3 of each
// 16, which is how the second product takes them, since a contraction may run
// over its index in any order as long as both operands agree. V^T wants 8
// tokens of one channel in a lane: the lane loads the same 8 (d = 128) or 4
// channels of its 8 tokens, one contiguous run per token across 16 lanes, and
// the transposition happens in the byte permutes that widen the codes.
// (Channel n of lane c belongs to matrix row c of the n-th product.)
//
// Bound: memory. The codes are read once; a tile costs 2 d / 16 matrix
// instructions per 16 rows, far below their rate.
//
// Number formats: int8 and e4m3 codes, and the pool's levels, are widened to
// binary16, where codes are exact (levels: rounded, 2^-12). Queries go to
// binary16 after division by a power of two per row (the row's largest
// becomes 2^14..2^15, so what is lost is below 2^-39 of it). Weights p * step
// go to binary16 (2^-12) after division by 2^E, E the wave's largest step
// exponent so far, times 2^12: the largest stays below 2^16 (m may lag the
// true maximum by kSlack), and weights down to 2^-26 of it keep all bits. A
// bf16 cache uses bf16 instructions, each p split into two bf16 terms, since
// one alone (2^-9) would show next to the output's own rounding.
//
// m is moved only when a tile's maximum passes it by kSlack (exponents of 2):
// most tiles then need no exchange between lanes and no rescaling.
#include "attend.h"
#include "codebook.h"
#include "kernels_common.h"

namespace kvc {
namespace {

constexpr int kDevBadHeader = 1, kDevBadPage = 32, kDevBadLength = 64;  // KVC_DEV_*
constexpr int kFmtBf16 = 0, kFmtInt8 = 1, kFmtFp8 = 2, kFmtPool = 3;
constexpr int kWaves = 4;
constexpr uint32_t kTile = 32;
constexpr uint32_t kMaxChunk = 4096;  // 32 tiles a wave: one page number of 16 tokens in each of 64 lanes
constexpr float kSlack = 3.0f;
constexpr int kWeightExp = 12;
constexpr float kNegInf = -__builtin_inff();

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct AttendParams {
    RowsDev q, out;
    float* lse;
    float* part;    // f32 sums [Hq * n][splits][d], then {m, l} [Hq * n][splits]
    int32_t* status;
    uint32_t n, H, Hq, group;   // sequences (or agents), kv heads, query heads, Hq / H
    uint32_t rows, row_blocks;  // query rows of one unit, workgroups of it
    uint32_t chunk, chunks;
    uint32_t splits, split0;    // parts of a row in all, and this launch's first
    uint32_t direct;            // one part: outputs are final
    float scale_log2;
    // pool
    const uint8_t* pool;
    PoolLayout lay;
    uint32_t L, T, layer;
    // pages
    const uint8_t* pages;
    const int32_t* table;
    uint64_t table_stride;
    const int32_t* lens;
    uint32_t table_cols, num_pages, page_shift;
    uint64_t page_bytes, steps;
};

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ f32x4 mfma_half(const u32x4& a, const u32x4& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c, 0,
                                                  0, 0);
}
__device__ __forceinline__ f32x4 mfma_bf16(const u32x4& a, const u32x4& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
}
template <int FMT>
__device__ __forceinline__ f32x4 mfma(const u32x4& a, const u32x4& b, const f32x4& c) {
    return FMT == kFmtBf16 ? mfma_bf16(a, b, c) : mfma_half(a, b, c);
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    half2_t r;
    r.x = (_Float16)lo;
    r.y = (_Float16)hi;
    return __builtin_bit_cast(uint32_t, r);
}

// Bytes b0, b1 (or b2, b3) of w, int8 codes with their sign bit flipped, to
// two binary16 codes: 0x64bb is 1024 + b, exact, and so is the difference.
template <bool HI>
__device__ __forceinline__ uint32_t widen_int8(uint32_t w) {
    const uint32_t u = __builtin_amdgcn_perm(0x64646464u, w, HI ? 0x04030402u : 0x04010400u);
    const half2_t bias = {(_Float16)1152.0f, (_Float16)1152.0f};
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, u) - bias);
}
template <bool HI>
__device__ __forceinline__ uint32_t widen_fp8(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.0f, HI));
}
template <int FMT, bool HI>
__device__ __forceinline__ uint32_t widen(uint32_t w) {
    return FMT == kFmtFp8 ? widen_fp8<HI>(w) : widen_int8<HI>(w);
}

// Level i of the value codes as binary16, and one byte (from bit `shift`) of
// levels first .. first + 3.
constexpr uint32_t level_half(int i) {
    const float pos[4] = {kLv0, kLv1, kLv2, kLv3};
    return __builtin_bit_cast(uint16_t, (_Float16)(i < 4 ? -pos[3 - i] : pos[i - 4]));
}
constexpr uint32_t level_bytes(int first, int shift) {
    uint32_t w = 0;
    for (int i = 0; i < 4; ++i) w |= (level_half(first + i) >> shift & 255u) << (8 * i);
    return w;
}

// What a lane loads of one tile: keys of tokens lane % 16 and 16 + lane % 16
// (its quarter of the channels), and of its 8 value tokens (4g + j, 16 + 4g + j)
// the channels of matrix rows lane % 16.
template <int FMT, int D>
struct Raw {
    static constexpr int KL = FMT == kFmtBf16 ? D / 32 : D / 64;  // 16-byte loads of a key row
    static constexpr int VW = FMT == kFmtBf16 ? D / 32 : D / 64;  // 4-byte words of a value row
    uint4 k[2][KL];
    uint32_t v[8][VW];
    float ks[8], vs[8];
};
template <int D>
struct Raw<kFmtPool, D> {
    uint4 k[2][D / 64];
    uint32_t v[8];   // three plane bytes (d = 128) or nibbles' bytes (d = 64)
    uint32_t vs[4];  // eight binary16 sizes
};

template <int W>
__device__ __forceinline__ void load_words(const uint8_t* a, uint32_t (&w)[W]) {
    if constexpr (W == 4) {
        const uint4 x = *reinterpret_cast<const uint4*>(a);
        w[0] = x.x;
        w[1] = x.y;
        w[2] = x.z;
        w[3] = x.w;
    } else if constexpr (W == 2) {
        const uint2 x = *reinterpret_cast<const uint2*>(a);
        w[0] = x.x;
        w[1] = x.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(a);
    }
}

__device__ __forceinline__ bool pool_header_ok(const AttendParams& p, uint32_t D) {
    const uint32_t* hd = reinterpret_cast<const uint32_t*>(p.pool);
    const uint64_t t = (uint64_t)hd[14] | ((uint64_t)hd[15] << 32);
    return hd[0] == kPoolMagic && hd[1] == (1u | (1u << 16)) && hd[2] == p.L && hd[3] == p.H && hd[4] == p.T &&
           hd[5] == D && t == p.lay.total;
}

// The sequence's length, within what its table's row holds.
__device__ __forceinline__ uint32_t length_of(const AttendParams& p, uint32_t b, bool tell) {
    const int32_t len = p.lens[b];
    const uint32_t most = p.table_cols << p.page_shift;
    if (len < 0 || (uint32_t)len > most) {
        if (tell && p.status) atomicOr(p.status, kDevBadLength);
        return len < 0 ? 0 : most;
    }
    return (uint32_t)len;
}

// Query row r (of the unit's rows) -> sequence and query head.
template <int FMT>
__device__ __forceinline__ void row_of(const AttendParams& p, uint32_t b, uint32_t h, uint32_t r, uint32_t& seq,
                                       uint32_t& qh) {
    if (FMT == kFmtPool) {
        seq = r / p.group;
        qh = h * p.group + r % p.group;
    } else {
        seq = b;
        qh = h * p.group + r;
    }
}

// In-place Walsh-Hadamard transform of the C channels of a thread and of the
// 16 threads (neighbouring lanes) that hold a row, Sylvester order.
template <int C>
__device__ __forceinline__ void fwht_row(float (&y)[C], uint32_t lane) {
#pragma unroll
    for (int h = 1; h < C; h *= 2) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            if ((i & h) == 0) {
                const float a = y[i], b = y[i + h];
                y[i] = a + b;
                y[i + h] = a - b;
            }
        }
    }
#pragma unroll
    for (int h = 1; h < 16; h *= 2) {
        const float s = (lane & h) ? -1.0f : 1.0f;
#pragma unroll
        for (int i = 0; i < C; ++i) y[i] = fmaf(s, y[i], __shfl_xor(y[i], h));
    }
}

template <int FMT, int D, int RT>
__global__ __launch_bounds__(kWaves* kWave) void attend_kernel(AttendParams p) {
    constexpr int KS = D / 32;   // key product steps
    constexpr int NC = D / 16;   // channels of a lane, value products
    constexpr bool HALF = FMT != kFmtBf16;
    using R = Raw<FMT, D>;
    const uint32_t lane = lane_id(), c = lane & 15, g = lane >> 4;
    const uint32_t wave = wave_uniform(threadIdx.x / kWave);

    // workgroup -> (row block, chunk, kv head, sequence); the row blocks of a
    // chunk, which read the same tokens, sit 8 workgroups apart: on one XCD
    uint32_t rb = 0, u = blockIdx.x;
    if (p.row_blocks > 1) {
        const uint32_t span = 8 * p.row_blocks;
        rb = (blockIdx.x % span) / 8;
        u = blockIdx.x / span * 8 + blockIdx.x % 8;
    }
    const uint32_t ck = u % p.chunks;
    const uint32_t h = u / p.chunks % p.H;
    const uint32_t b = u / p.chunks / p.H;
    if (b >= (FMT == kFmtPool ? 1u : p.n)) return;  // the padding of the last 8

    uint32_t len;
    if (FMT == kFmtPool) {
        if (!pool_header_ok(p, D)) {
            if (threadIdx.x == 0 && p.status) atomicOr(p.status, kDevBadHeader);
            return;
        }
        len = p.T;
    } else {
        len = wave_uniform(length_of(p, b, threadIdx.x == 0 && ck == 0 && h == 0 && rb == 0));
    }
    const uint32_t begin = ck * p.chunk;
    if (begin >= len && !(p.direct && ck == 0)) return;
    const uint32_t end = len - begin < p.chunk ? len : begin + p.chunk;  // begin <= len here

    // page numbers of this wave's 16-token runs: run i of tile t in lane 2t + i
    uint32_t my_page = 0;
    if (FMT != kFmtPool) {
        const uint32_t t = begin + ((lane >> 1) * kWaves + wave) * kTile + (lane & 1) * 16;
        if (t < end) {
            const int32_t pg = p.table[b * p.table_stride + (t >> p.page_shift)];
            const bool ok = (uint32_t)pg < p.num_pages;
            if (!ok && p.status) atomicOr(p.status, kDevBadPage);
            my_page = ok ? (uint32_t)pg : 0;
        }
    }

    // queries: row 16 rt + c, channels as the key loads have them
    u32x4 qf[RT][KS];
    float qscale[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const uint32_t r = (rb * RT + rt) * 16 + c;
        uint32_t w[KS][4];
        uint32_t seq, qh;
        row_of<FMT>(p, b, h, r < p.rows ? r : 0, seq, qh);
        const uint8_t* qp = reinterpret_cast<const uint8_t*>(p.q.data + (uint64_t)seq * p.q.ts + (uint64_t)qh * p.q.hs);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const uint32_t ch = HALF ? (s / 2) * 64 + g * 16 + (s % 2) * 8 : s * 32 + g * 8;
            load_words(qp + 2 * ch, w[s]);
            if (r >= p.rows) w[s][0] = w[s][1] = w[s][2] = w[s][3] = 0;
        }
        qscale[rt] = p.scale_log2;
        if (HALF) {
            uint32_t m = 0;
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t lo = w[s][i] & 0x7FFFu, hi = (w[s][i] >> 16) & 0x7FFFu;
                    m = lo > m ? lo : m;
                    m = hi > m ? hi : m;
                }
            uint32_t o = __shfl_xor(m, 16);
            m = o > m ? o : m;
            o = __shfl_xor(m, 32);
            m = o > m ? o : m;
            // largest magnitude to [2^14, 2^15); Inf and NaN stay what they are
            const int e = (m == 0 || m >= 0x7F80u) ? 0 : 15 - __builtin_amdgcn_frexp_expf(__uint_as_float(m << 16));
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    qf[rt][s][i] = pack_half2(__builtin_amdgcn_ldexpf(bf16_lo(w[s][i]), e),
                                              __builtin_amdgcn_ldexpf(bf16_hi(w[s][i]), e));
            qscale[rt] = __builtin_amdgcn_ldexpf(qscale[rt], -e);
        } else {
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) qf[rt][s][i] = w[s][i];
        }
    }
    if (FMT == kFmtPool) {
        const float step = reinterpret_cast<const float*>(p.pool + p.lay.k_scale)[p.layer];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) qscale[rt] *= step;
    }

    // running state
    f32x4 o[RT][NC];
    float m[RT], mu[RT], l[RT];
    int E = -1000;  // exponent taken out of the weights (HALF)
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        m[rt] = kNegInf;
        mu[rt] = 0.0f;
        l[rt] = 0.0f;
#pragma unroll
        for (int n = 0; n < NC; ++n) o[rt][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    const uint64_t vec0 = FMT == kFmtPool ? ((uint64_t)p.layer * p.H + h) * p.T : 0;  // the head's first vector
    const auto load = [&](uint32_t t0, uint32_t it, R& x) {
        if constexpr (FMT == kFmtPool) {
            const uint64_t vec = vec0 + t0;
            const uint32_t last = p.T - t0 - 1;  // tokens behind the last are the last again (masked below)
            const uint8_t* kb = p.pool + p.lay.k_codes + vec * D;
            const uint8_t* vb = p.pool + p.lay.v_codes + vec * (3 * D / 8);
            const uint8_t* sb = p.pool + p.lay.v_scale + vec * 2;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t t = 16 * i + c < last ? 16 * i + c : last;
#pragma unroll
                for (int s = 0; s < D / 64; ++s)
                    x.k[i][s] = *reinterpret_cast<const uint4*>(kb + t * D + 64 * s + 16 * g);
            }
            const uint32_t at = D == 128 ? c : c >> 1;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t t0j = (j < 4 ? 0 : 16) + 4 * g + (j & 3);
                const uint32_t t = t0j < last ? t0j : last;
                const uint8_t* a = vb + t * (3 * D / 8) + at;
                x.v[j] = (uint32_t)a[0] | (uint32_t)a[D / 8] << 8 | (uint32_t)a[2 * D / 8] << 16;
                const uint32_t sz = *reinterpret_cast<const uint16_t*>(sb + 2 * t);
                if (j & 1)
                    x.vs[j >> 1] |= sz << 16;
                else
                    x.vs[j >> 1] = sz;
            }
        } else {
            constexpr uint32_t ROW = FMT == kFmtBf16 ? 2 * D : D;
            const uint32_t P = 1u << p.page_shift;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t pg = __builtin_amdgcn_readlane(my_page, (2 * it + i) & 63);
                const uint8_t* pb = p.pages + (uint64_t)pg * p.page_bytes;
                const uint32_t at = (t0 + 16 * i) & (P - 1);
                const uint32_t kl = h * P + at, vl = (p.H + h) * P + at;  // rows inside the page
                const uint8_t* kb = pb + (uint64_t)kl * ROW;
                const uint8_t* vb = pb + (uint64_t)vl * ROW;
#pragma unroll
                for (int s = 0; s < R::KL; ++s)
                    x.k[i][s] = *reinterpret_cast<const uint4*>(kb + c * ROW + 64 * s + 16 * g);
#pragma unroll
                for (int j = 0; j < 4; ++j) load_words(vb + (4 * g + j) * ROW + c * (ROW / 16), x.v[4 * i + j]);
                if (FMT != kFmtBf16) {
                    const float4 a = *reinterpret_cast<const float4*>(pb + p.steps + (uint64_t)(kl + 4 * g) * 4);
                    const float4 w = *reinterpret_cast<const float4*>(pb + p.steps + (uint64_t)(vl + 4 * g) * 4);
                    x.ks[4 * i] = a.x;
                    x.ks[4 * i + 1] = a.y;
                    x.ks[4 * i + 2] = a.z;
                    x.ks[4 * i + 3] = a.w;
                    x.vs[4 * i] = w.x;
                    x.vs[4 * i + 1] = w.y;
                    x.vs[4 * i + 2] = w.z;
                    x.vs[4 * i + 3] = w.w;
                }
            }
        }
    };

    const auto tile = [&](uint32_t t0, R& x) {
        const uint32_t live = end - t0;  // tokens of this tile that count, if below 32
        // key operands
        u32x4 kf[2][KS];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                if (HALF) {
                    const uint4& y = x.k[i][s / 2];
                    uint32_t a = s % 2 ? y.z : y.x, d = s % 2 ? y.w : y.y;
                    if (FMT != kFmtFp8) {
                        a ^= 0x80808080u;
                        d ^= 0x80808080u;
                    }
                    constexpr int F = FMT == kFmtFp8 ? kFmtFp8 : kFmtInt8;
                    kf[i][s] = u32x4{widen<F, false>(a), widen<F, true>(a), widen<F, false>(d), widen<F, true>(d)};
                } else {
                    const uint4& y = x.k[i][s];
                    kf[i][s] = u32x4{y.x, y.y, y.z, y.w};
                }
            }
        }
        // value operands: token pairs of one channel
        u32x4 vf[NC];
        float vs[8];
        if constexpr (FMT == kFmtPool) {
            // plane words: byte j of pl[half][q] is plane q of token j
            uint32_t pl[2][3];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int q = 0; q < 3; ++q) {
                    const uint32_t lo = __builtin_amdgcn_perm(x.v[4 * i + 1], x.v[4 * i], 0x0C0C0400u + 0x0101u * q);
                    const uint32_t hi = __builtin_amdgcn_perm(x.v[4 * i + 3], x.v[4 * i + 2], 0x04000C0Cu + 0x01010000u * q);
                    pl[i][q] = lo | hi;
                    if (D == 64) pl[i][q] = pl[i][q] >> ((c & 1) * 4) & 0x0F0F0F0Fu;
                }
            }
            // levels as binary16: a byte table of the low and of the high halves
            constexpr uint32_t l0 = level_bytes(0, 0), l1 = level_bytes(4, 0);
            constexpr uint32_t h0 = level_bytes(0, 8), h1 = level_bytes(4, 8);
#pragma unroll
            for (int n = 0; n < NC; ++n) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t sel = pl[i][0] >> n & 0x01010101u;
                    sel |= (n >= 1 ? pl[i][1] >> (n >= 1 ? n - 1 : 0) : pl[i][1] << 1) & 0x02020202u;
                    sel |= (n >= 2 ? pl[i][2] >> (n >= 2 ? n - 2 : 0) : pl[i][2] << (n >= 2 ? 0 : 2 - n)) & 0x04040404u;
                    const uint32_t lo = __builtin_amdgcn_perm(l1, l0, sel), hi = __builtin_amdgcn_perm(h1, h0, sel);
                    vf[n][2 * i] = __builtin_amdgcn_perm(hi, lo, 0x05010400u);
                    vf[n][2 * i + 1] = __builtin_amdgcn_perm(hi, lo, 0x07030602u);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const half2_t s2 = __builtin_bit_cast(half2_t, x.vs[j]);
                vs[2 * j] = (float)s2.x;
                vs[2 * j + 1] = (float)s2.y;
            }
        } else {
            if (live < kTile) {
                // rows behind the end may hold anything: NaN times a weight of 0 would stay
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const bool ok = (j < 4 ? 0 : 16) + 4 * g + (j & 3) < live;
#pragma unroll
                    for (int w = 0; w < R::VW; ++w) x.v[j][w] = ok ? x.v[j][w] : 0;
                    if (FMT != kFmtBf16) x.vs[j] = ok ? x.vs[j] : 0.0f;
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // token pair (2j, 2j + 1)
#pragma unroll
                for (int w = 0; w < R::VW; ++w) {
                    uint32_t a = x.v[2 * j][w], d = x.v[2 * j + 1][w];
                    if constexpr (FMT == kFmtBf16) {
                        vf[2 * w][j] = __builtin_amdgcn_perm(d, a, 0x05040100u);
                        vf[2 * w + 1][j] = __builtin_amdgcn_perm(d, a, 0x07060302u);
                    } else {
                        if (FMT == kFmtInt8) {
                            a ^= 0x80808080u;
                            d ^= 0x80808080u;
                        }
                        const uint32_t lo = __builtin_amdgcn_perm(d, a, 0x05010400u);
                        const uint32_t hi = __builtin_amdgcn_perm(d, a, 0x07030602u);
                        vf[4 * w][j] = widen<FMT, false>(lo);
                        vf[4 * w + 1][j] = widen<FMT, true>(lo);
                        vf[4 * w + 2][j] = widen<FMT, false>(hi);
                        vf[4 * w + 3][j] = widen<FMT, true>(hi);
                    }
                }
            }
            if (FMT != kFmtBf16) {
#pragma unroll
                for (int j = 0; j < 8; ++j) vs[j] = x.vs[j];
            }
        }
        if (HALF) {
            // step exponents: all weights are divided by 2^E
            float big = vs[0];
#pragma unroll
            for (int j = 1; j < 8; ++j) big = fmaxf(big, vs[j]);
            const int e = big > 0.0f ? __builtin_amdgcn_frexp_expf(big) : -1000;
            if (__ballot(e > E) != 0) {
                int ne = e > E ? e : E;
                int other = __shfl_xor(ne, 16);
                ne = other > ne ? other : ne;
                other = __shfl_xor(ne, 32);
                ne = other > ne ? other : ne;
                if (E > -1000) {
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                        for (int n = 0; n < NC; ++n)
#pragma unroll
                            for (int r = 0; r < 4; ++r) o[rt][n][r] = __builtin_amdgcn_ldexpf(o[rt][n][r], E - ne);
                }
                E = ne;
            }
            const int shift = E > -1000 ? kWeightExp - E : 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) vs[j] = __builtin_amdgcn_ldexpf(vs[j], shift);
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            f32x4 s[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                s[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int k = 0; k < KS; ++k) s[i] = mfma<FMT>(kf[i][k], qf[rt][k], s[i]);
            }
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                y[j] = s[j >> 2][j & 3] * qscale[rt];
                if constexpr (FMT == kFmtInt8 || FMT == kFmtFp8) y[j] *= x.ks[j];
            }
            if (live < kTile) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    y[j] = (j < 4 ? 0 : 16) + 4 * g + (j & 3) < live ? y[j] : kNegInf;
            }
            float top = y[0];
#pragma unroll
            for (int j = 1; j < 8; ++j) top = fmaxf(top, y[j]);
            if (__ballot(top > m[rt] + kSlack) != 0) {
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                const float nm = fmaxf(m[rt], top);
                const float a = nm == kNegInf ? 1.0f : exp2_fast(m[rt] - nm);
                m[rt] = nm;
                mu[rt] = nm == kNegInf ? 0.0f : nm;
                l[rt] *= a;
#pragma unroll
                for (int n = 0; n < NC; ++n) o[rt][n] *= a;
            }
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float e = exp2_fast(y[j] - mu[rt]);
                l[rt] += e;
                w[j] = HALF ? e * vs[j] : e;
            }
            if (HALF) {
                u32x4 pf;
#pragma unroll
                for (int j = 0; j < 4; ++j) pf[j] = pack_half2(w[2 * j], w[2 * j + 1]);
#pragma unroll
                for (int n = 0; n < NC; ++n) o[rt][n] = mfma_half(vf[n], pf, o[rt][n]);
            } else {
                u32x4 hi, lo;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    hi[j] = pack_bf16x2(w[2 * j], w[2 * j + 1]);
                    lo[j] = pack_bf16x2(w[2 * j] - bf16_lo(hi[j]), w[2 * j + 1] - bf16_hi(hi[j]));
                }
#pragma unroll
                for (int n = 0; n < NC; ++n) o[rt][n] = mfma_bf16(vf[n], lo, mfma_bf16(vf[n], hi, o[rt][n]));
            }
        }
    };

    {
        uint32_t it = 0;
        for (uint32_t t0 = begin + wave * kTile; t0 < end; t0 += kWaves * kTile, ++it) {
            R x;
            load(t0, it, x);
            tile(t0, x);
        }
    }

    // ---- join the waves: m and l first, then the sums, 16 rows at a time
    __shared__ float ml[kWaves][RT * 16][2];
    __shared__ float os[kWaves][16][D + 4];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        float s = l[rt];
        s += __shfl_xor(s, 16);
        s += __shfl_xor(s, 32);
        if (g == 0) {
            ml[wave][rt * 16 + c][0] = m[rt];
            ml[wave][rt * 16 + c][1] = s;
        }
    }
    __syncthreads();
    const uint32_t row = threadIdx.x / 16, ch = threadIdx.x % 16 * NC;  // the thread's part of the outputs
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        float M = ml[0][rt * 16 + c][0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) M = fmaxf(M, ml[w][rt * 16 + c][0]);
        const float Mu = M == kNegInf ? 0.0f : M;
        float a = exp2_fast(m[rt] - Mu);
        const int sh = HALF && E > -1000 ? E - kWeightExp : 0;
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                float v = o[rt][n][r];
                if (HALF) v = __builtin_amdgcn_ldexpf(v, sh);
                os[wave][c][(4 * g + r) * NC + n] = v * a;
            }
        __syncthreads();
        const uint32_t r = (rb * RT + rt) * 16 + row;
        float Mr = ml[0][rt * 16 + row][0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) Mr = fmaxf(Mr, ml[w][rt * 16 + row][0]);
        const float Mru = Mr == kNegInf ? 0.0f : Mr;
        float total = 0.0f, y[NC];
#pragma unroll
        for (int n = 0; n < NC; ++n) y[n] = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            total = fmaf(ml[w][rt * 16 + row][1], exp2_fast(ml[w][rt * 16 + row][0] - Mru), total);
#pragma unroll
            for (int n = 0; n < NC; ++n) y[n] += os[w][row][ch + n];
        }
        if (FMT == kFmtPool) {
            fwht_row<NC>(y, lane);
            const float k = D == 128 ? 0.08838834764831845f : 0.125f;  // 1 / sqrt(d)
#pragma unroll
            for (int n = 0; n < NC; ++n) y[n] *= k;
        }
        if (r < p.rows) {
            uint32_t seq, qh;
            row_of<FMT>(p, b, h, r, seq, qh);
            const uint64_t at = (uint64_t)seq * p.Hq + qh;
            if (p.direct) {
                // a row without tokens: zeros, and ln 0
                const float inv = total == 0.0f ? 0.0f : 1.0f / total;
                uint16_t* to = p.out.data + (uint64_t)seq * p.out.ts + (uint64_t)qh * p.out.hs + ch;
                uint32_t w[NC / 2];
#pragma unroll
                for (int n = 0; n < NC / 2; ++n) w[n] = pack_bf16x2(y[2 * n] * inv, y[2 * n + 1] * inv);
                if constexpr (NC == 8)
                    *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
                else
                    *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
                if (p.lse && threadIdx.x % 16 == 0) p.lse[at] = (Mr + log2f(total)) * 0.69314718055994531f;
            } else {
                const uint64_t part = at * p.splits + p.split0 + ck;
                float* to = p.part + part * D + ch;
#pragma unroll
                for (int n = 0; n < NC; n += 4) *reinterpret_cast<f32x4*>(to + n) = f32x4{y[n], y[n + 1], y[n + 2], y[n + 3]};
                if (threadIdx.x % 16 == 0) {
                    float* t2 = p.part + (uint64_t)p.n * p.Hq * p.splits * D + part * 2;
                    t2[0] = Mr;
                    t2[1] = total;
                }
            }
        }
        __syncthreads();
    }
}

// Joins the parts of a row: one wave per row, d / 64 channels a lane.
struct JoinParams {
    RowsDev out;
    float* lse;
    const float* part;
    uint32_t n, Hq, splits;
    uint32_t pool_splits;     // parts that are always there
    uint32_t chunk;           // tokens of a tail's part
    AttendParams src;         // header and lengths
};

template <int D>
__global__ __launch_bounds__(kBlockThreads) void attend_join_kernel(JoinParams p) {
    constexpr int C = D / 64;
    const uint32_t lane = lane_id();
    const uint64_t row = (uint64_t)blockIdx.x * (kBlockThreads / kWave) + wave_uniform(threadIdx.x / kWave);
    if (row >= (uint64_t)p.n * p.Hq) return;
    if (p.src.pool && !pool_header_ok(p.src, D)) return;
    const uint32_t seq = (uint32_t)(row / p.Hq), qh = (uint32_t)(row % p.Hq);
    uint32_t parts = p.pool_splits;
    if (p.src.table) parts += (length_of(p.src, seq, false) + p.chunk - 1) / p.chunk;
    const float* o = p.part + row * p.splits * D;
    const float* ml = p.part + (uint64_t)p.n * p.Hq * p.splits * D + row * p.splits * 2;
    float M = kNegInf;
    for (uint32_t s = lane; s < parts; s += kWave) M = fmaxf(M, ml[2 * s]);
#pragma unroll
    for (int x = 1; x < 64; x *= 2) M = fmaxf(M, __shfl_xor(M, x));
    const float Mu = M == kNegInf ? 0.0f : M;
    float total = 0.0f, y[C];
#pragma unroll
    for (int i = 0; i < C; ++i) y[i] = 0.0f;
    for (uint32_t s = 0; s < parts; ++s) {
        const float a = exp2_fast(ml[2 * s] - Mu);
        total = fmaf(ml[2 * s + 1], a, total);
#pragma unroll
        for (int i = 0; i < C; ++i) y[i] = fmaf(o[(uint64_t)s * D + C * lane + i], a, y[i]);
    }
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    uint16_t* to = p.out.data + (uint64_t)seq * p.out.ts + (uint64_t)qh * p.out.hs;
    if constexpr (C == 2)
        reinterpret_cast<uint32_t*>(to)[lane] = pack_bf16x2(y[0] * inv, y[1] * inv);
    else
        to[lane] = (uint16_t)pack_bf16x2(y[0] * inv, 0.0f);
    if (p.lse && lane == 0) p.lse[row] = (M + log2f(total)) * 0.69314718055994531f;
}

template <int FMT, int D>
hipError_t launch_rt(uint32_t rt, uint32_t grid, const AttendParams& p, hipStream_t stream) {
    return launch_kernel(rt == 1   ? attend_kernel<FMT, D, 1>
                         : rt == 2 ? attend_kernel<FMT, D, 2>
                                   : attend_kernel<FMT, D, 4>,
                         dim3(grid), dim3(kWaves * kWave), stream, p);
}

template <int FMT>
hipError_t launch_source(uint32_t d, const AttendPlan& plan, AttendParams& p, uint32_t units, hipStream_t stream) {
    p.rows = plan.rows;
    p.row_blocks = plan.row_blocks;
    p.chunk = plan.chunk;
    p.chunks = plan.chunks;
    uint64_t blocks = (uint64_t)units * plan.chunks;
    if (plan.row_blocks > 1) blocks = (blocks + 7) / 8 * 8 * plan.row_blocks;
    return d == 64 ? launch_rt<FMT, 64>(plan.rt, (uint32_t)blocks, p, stream)
                   : launch_rt<FMT, 128>(plan.rt, (uint32_t)blocks, p, stream);
}

uint32_t tiles_of(uint32_t rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }

AttendPlan make_plan(uint64_t units, uint32_t rows, uint64_t max_tokens) {
    AttendPlan a;
    a.rows = rows;
    a.rt = tiles_of(rows);
    a.row_blocks = (rows + 16 * a.rt - 1) / (16 * a.rt);
    const uint64_t groups = units * a.row_blocks;
    uint64_t chunk = max_tokens * groups / 1024;
    chunk = chunk < 256 ? 256 : (chunk + 127) / 128 * 128;
    a.chunk = (uint32_t)(chunk > kMaxChunk ? kMaxChunk : chunk);
    a.chunks = (uint32_t)((max_tokens + a.chunk - 1) / a.chunk);
    if (a.chunks == 0) a.chunks = 1;
    return a;
}

}  // namespace

AttendPlan page_attend_plan(uint32_t n_seqs, uint32_t H, uint32_t Hq, uint64_t max_tokens) {
    return make_plan((uint64_t)n_seqs * H, Hq / H, max_tokens);
}

AttendPlan pool_attend_plan(uint32_t H, uint32_t n_agents, uint32_t Hq, uint32_t T) {
    return make_plan(H, n_agents * (Hq / H), T);
}

hipError_t launch_attend(const AttendArgs& a, hipStream_t stream) {
    AttendParams p{};
    p.q = a.q;
    p.out = a.out;
    p.lse = a.lse;
    p.part = a.ws;
    p.status = a.status;
    p.n = a.n;
    p.H = a.H;
    p.Hq = a.Hq;
    p.group = a.Hq / a.H;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    AttendPlan pool_plan{}, page_plan{};
    const bool has_pool = a.pool != nullptr, has_pages = a.tail.table != nullptr;
    if (has_pool) {
        pool_plan = pool_attend_plan(a.H, a.n, a.Hq, a.T);
        p.pool = a.pool;
        p.lay = pool_layout(a.L, a.H, a.T, a.d);
        p.L = a.L;
        p.T = a.T;
        p.layer = a.layer;
    }
    if (has_pages) {
        const PageLayout& lay = a.tail.lay;
        page_plan = page_attend_plan(a.n, a.H, a.Hq, (uint64_t)a.tail.table_cols * lay.P);
        p.pages = a.tail.pages;
        p.table = a.tail.table;
        p.table_stride = a.tail.table_stride;
        p.lens = a.tail.lens;
        p.table_cols = a.tail.table_cols;
        p.num_pages = lay.num_pages;
        p.page_shift = 31 - __builtin_clz(lay.P);
        p.page_bytes = lay.page_bytes;
        p.steps = lay.steps;
    }
    p.splits = (has_pool ? pool_plan.chunks : 0) + (has_pages ? page_plan.chunks : 0);
    p.direct = p.splits == 1;
    hipError_t e = hipSuccess;
    if (has_pool) e = launch_source<kFmtPool>(a.d, pool_plan, p, a.H, stream);
    if (has_pages && e == hipSuccess) {
        p.split0 = has_pool ? pool_plan.chunks : 0;
        const uint32_t units = a.n * a.H;
        e = a.tail.lay.format == 0   ? launch_source<kFmtBf16>(a.d, page_plan, p, units, stream)
            : a.tail.lay.format == 1 ? launch_source<kFmtInt8>(a.d, page_plan, p, units, stream)
                                     : launch_source<kFmtFp8>(a.d, page_plan, p, units, stream);
    }
    if (p.direct || e != hipSuccess) return e;
    JoinParams j{};
    j.out = a.out;
    j.lse = a.lse;
    j.part = a.ws;
    j.n = a.n;
    j.Hq = a.Hq;
    j.splits = p.splits;
    j.pool_splits = has_pool ? pool_plan.chunks : 0;
    j.chunk = has_pages ? page_plan.chunk : 1;
    j.src = p;
    const uint64_t rows = (uint64_t)a.n * a.Hq;
    return launch_kernel(a.d == 64 ? attend_join_kernel<64> : attend_join_kernel<128>,
                         dim3((uint32_t)((rows + 3) / 4)), dim3(kBlockThreads), stream, j);
}

}  // namespace kvc
