// prompt_kernels.hip - attention of many new tokens of each sequence over its
// pages (a prompt, a part of one, drafted tokens), for gfx950.
//
// The query rows of a sequence and kv head are its new tokens times the query heads
// that share the kv head, token by token. A workgroup takes 128 of them, 32 a wave, and
// walks the tokens that they see in tiles of 64, with one pass over the data
// (running maximum m and sum l):
//     S^T = K Q^T           32x32x16 matrix instructions, tokens x rows
//     p = exp2(f S - m)     in the lanes that hold S
//     O^T += V^T p^T        32x32x16, channels x rows
// In both products a lane's column is one query row (lane % 32), shared with lane + 32,
// so m and l are its own registers. S^T leaves a lane with tokens 8j + 4 (lane / 32) +
// 0..3, and the second product takes its tokens in that order: the transposed LDS read
// gives four tokens of one channel to a lane, so V stays in LDS as it is in memory.
#include "attend.h"
#include "kernels_common.h"
#include "page_codes.h"

#include <type_traits>

namespace kvc {
namespace {

constexpr int kDevBadPage = 32, kDevBadLength = 64, kDevBadStart = 128;  // KVC_DEV_*
constexpr uint32_t kRows = 128;    // of a workgroup
constexpr uint32_t kTokens = 64;   // of a tile
constexpr uint32_t kRun = 16;      // tokens that lie in one page: a wave fetches one run of each tile
constexpr int kWavesOf = 4;
constexpr float kSlack = 3.0f;     // m moves when a tile's maximum passes it by this (powers of two)
constexpr int kWeightExp = 12;     // binary16 weights: the largest stays below 2^(12 + 3 + 1)
constexpr float kNegInf = -__builtin_inff();
constexpr bool half_products(int fmt) { return fmt == kPageInt8 || fmt == kPageFp8; }

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
#define KVC_LDS __attribute__((address_space(3)))

struct PromptParams {
    RowsDev q, out;
    float* lse;
    int32_t* status;
    const int32_t *starts, *lens, *table;
    const uint8_t* pages;
    uint64_t table_stride, page_bytes, steps;
    uint32_t n, rows, H, Hq, group;
    uint32_t table_cols, num_pages, page_shift;
    uint32_t window, sinks;
    uint32_t splits;
    float scale_log2;
    float* part;  // of each split and row: sums [splits][rows * Hq][d], then {m, l} [splits][rows * Hq][2]
};

template <int FMT>
__device__ __forceinline__ f32x16 mfma(const u32x4& a, const u32x4& b, const f32x16& c) {
    if constexpr (half_products(FMT))
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// Over the two lanes that hold a query row, in both.
template <class T, class F>
__device__ __forceinline__ T over_pair(T v, F join) {
    const uint32_t a = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane32_swap(a, a, false, false);
    return join(__builtin_bit_cast(T, (uint32_t)r[0]), __builtin_bit_cast(T, (uint32_t)r[1]));
}

// Sum over the wave's lanes up to this one.
__device__ __forceinline__ uint32_t scan_lanes(uint32_t v) {
    const auto step = [&](auto ctrl, auto rows) {
        v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, decltype(rows)::value, 0xF, false);
    };
    using All = std::integral_constant<int, 0xF>;
    step(std::integral_constant<int, 0x111>{}, All{});  // from 1, 2, 4, 8 lanes before, in the row
    step(std::integral_constant<int, 0x112>{}, All{});
    step(std::integral_constant<int, 0x114>{}, All{});
    step(std::integral_constant<int, 0x118>{}, All{});
    step(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{});  // rows 0, 2 to 1, 3
    step(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xC>{});  // half 0 to 1
    return v;
}

// A tile in LDS holds rows of D 16-bit numbers, a token each, in chunks of 16 bytes, whose places are
// changed inside a row so that the lanes of one LDS cycle meet in no bank: of K, which 16 lanes read at one
// chunk of 16 tokens, by the token; of V, of which 32 lanes read 64 bytes of 4 tokens, by the token in runs of 64 bytes.
template <int D>
__device__ __forceinline__ uint32_t place_k(uint32_t token, uint32_t chunk) {
    return token * (2 * D) + ((chunk ^ (D == 128 ? token & 15 : token >> 1 & 7)) << 4);
}
template <int D>
__device__ __forceinline__ uint32_t place_v(uint32_t token, uint32_t chunk) {
    return token * (2 * D) + ((chunk ^ (D == 128 ? (token & 3) << 2 : (token >> 1 & 1) << 2)) << 4);
}

// 16 bytes of each lane from memory to LDS, at lds + 16 * lane.
__device__ __forceinline__ void fetch16(const uint8_t* from, uint8_t* lds) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(uint64_t)from, (KVC_LDS void*)lds, 16, 0, 0);
}

template <int FMT, int D>
struct Tile {
    static constexpr uint32_t kBytes = kTokens * D * 2;  // of keys, and of values
    alignas(16) uint8_t kv[2][2][kBytes];                // [buffer][keys, values]
    float steps[half_products(FMT) ? 2 : 1][2][half_products(FMT) ? kTokens : 1];
};

template <int FMT, int D>
__global__ __launch_bounds__(kWavesOf* kWave, 2) void prompt_kernel(PromptParams p) {
    fetch_arguments<sizeof(PromptParams)>();
    constexpr bool HALF = half_products(FMT);
    constexpr int KS = D / 16, CB = D / 32;
    __shared__ Tile<FMT, D> sh;
    const uint32_t lane = lane_id(), wave = wave_uniform(threadIdx.x / kWave);
    const uint32_t col = lane & 31, hi = lane >> 5;

    // ---- the block of rows: sequences and their blocks from the last to the first, so that the longest come first
    const uint32_t h = blockIdx.x % p.H, rest = blockIdx.x / p.H;
    const uint32_t split = rest % p.splits, block = rest / p.splits;
    uint32_t b = 0, row0 = 0, first = 0, m_rows = 0;  // sequence, first row of the block, first token's row, new tokens
    {
        uint32_t before = 0;
        bool found = false;
        for (uint32_t base = 0; base < p.n; base += kWave) {
            const bool live = base + lane < p.n;
            const uint32_t s = live ? p.n - 1 - base - lane : 0;
            const int32_t a = p.starts[s], e = p.starts[s + 1];
            const bool bad = a < 0 || e < a || (uint32_t)e > p.rows;
            if (live && bad && p.status) atomicOr(p.status, kDevBadStart);
            const uint32_t m = live && !bad ? e - a : 0;
            const uint32_t nb = (m * p.group + kRows - 1) / kRows;
            const uint32_t up = scan_lanes(nb);
            const uint32_t all = __builtin_amdgcn_readlane(up, 63);
            if (block < before + all) {
                const int at = __builtin_popcountll(__ballot(before + up <= block));
                b = __builtin_amdgcn_readlane(s, at);
                first = __builtin_amdgcn_readlane(a, at);
                m_rows = __builtin_amdgcn_readlane(m, at);
                row0 = (before + __builtin_amdgcn_readlane(up, at) - 1 - block) * kRows;
                found = true;
                break;
            }
            before += all;
        }
        if (!found) return;
    }
    const uint32_t unit_rows = m_rows * p.group;
    const uint32_t nrows = unit_rows - row0 < kRows ? unit_rows - row0 : kRows;
    const int32_t given = p.lens[b];
    const uint32_t most = p.table_cols << p.page_shift;
    const int32_t len = given < 0 ? 0 : (uint32_t)given > most ? (int32_t)most : given;
    if (len != given && p.status && threadIdx.x == 0) atomicOr(p.status, kDevBadLength);

    // ---- what its rows see: tokens below `sunk` and from lo to end, in tiles; tile i starts at start_of(i)
    const int32_t base_pos = len - (int32_t)m_rows;
    const int32_t pos_lo = base_pos + (int32_t)(row0 / p.group), pos_hi = base_pos + (int32_t)((row0 + nrows - 1) / p.group);
    const uint32_t end = pos_hi < 0 ? 0 : pos_hi + 1;
    const uint32_t lo = p.window && pos_lo >= 0 && (uint32_t)pos_lo >= p.window ? pos_lo - p.window + 1 : 0;
    const uint32_t sunk = p.sinks < lo ? p.sinks : lo;
    const uint32_t tiles0 = (sunk + kTokens - 1) / kTokens;
    const uint32_t from = lo / kTokens > tiles0 ? lo / kTokens : tiles0;
    const uint32_t tiles = tiles0 + ((end + kTokens - 1) / kTokens > from ? (end + kTokens - 1) / kTokens - from : 0);
    const auto start_of = [&](uint32_t i) { return (i < tiles0 ? i : i - tiles0 + from) * kTokens; };
    const uint32_t i0 = (uint32_t)((uint64_t)tiles * split / p.splits), i1 = (uint32_t)((uint64_t)tiles * (split + 1) / p.splits);

    // ---- this lane's row; a lane without one takes the block's last, which is not written
    const uint32_t my_row = wave * 32 + col;
    const bool has_row = my_row < nrows;
    const uint32_t R = row0 + (has_row ? my_row : nrows - 1);
    const uint32_t tok = R / p.group, qh = h * p.group + R % p.group;
    const int32_t pos = base_pos + (int32_t)tok;
    const bool works = wave * 32 < nrows;  // uniform
    // positions of the wave's rows
    const int32_t wave_lo = __builtin_amdgcn_readlane(pos, 0), wave_hi = __builtin_amdgcn_readlane(pos, 31);

    // ---- queries
    u32x4 qf[KS];
    float f = fabsf(p.scale_log2);
    f = fmaxf(f, 1e-45f);  // of a scale of 0: all logits alike, and -inf stays what it is
    {
        const uint16_t* qp = p.q.data + (uint64_t)(first + tok) * p.q.ts + (uint64_t)qh * p.q.hs + 8 * hi;
#pragma unroll
        for (int s = 0; s < KS; ++s) qf[s] = *reinterpret_cast<const u32x4*>(qp + 16 * s);
        if constexpr (HALF) {
            // to binary16: the row's largest magnitude to [2^14, 2^15), by 2^112 at most; Inf and NaN stay what they are
            uint32_t big = 0;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const uint32_t y = magnitude8(make_uint4(qf[s].x, qf[s].y, qf[s].z, qf[s].w));
                big = y > big ? y : big;
            }
            big = over_pair(big, [](uint32_t a, uint32_t c) { return a > c ? a : c; });
            int e = (big == 0 || big >= 0x7F80u) ? 0 : 15 - __builtin_amdgcn_frexp_expf(__uint_as_float(big << 16));
            e = e < 112 ? e : 112;
            const float up = copysignf(__builtin_amdgcn_ldexpf(1.0f, e), p.scale_log2);
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) qf[s][i] = pack_half2(bf16_lo(qf[s][i]) * up, bf16_hi(qf[s][i]) * up);
            f = fmaxf(__builtin_amdgcn_ldexpf(f, -e), 1e-45f);
        } else {
            const uint32_t turn = p.scale_log2 < 0.0f ? 0x80008000u : 0;
#pragma unroll
            for (int s = 0; s < KS; ++s) qf[s] ^= turn;
        }
    }

    // ---- tiles from memory: wave w fetches tokens 16 w .. 16 w + 15 of keys and values, one run, from one page. Tokens
    // that no row sees may hold anything, NaN too, which times a weight of 0 would stay: a token that is seen takes
    // their place, of the run if it has one, else the last of all.
    const auto needed = [&](uint32_t t) { return (t < end) & ((t < sunk) | (t + kRun > lo)); };
    const auto run_of = [&](uint32_t i) {
        const uint32_t t = start_of(i) + kRun * wave;
        return needed(t) ? t : (end - 1) & ~(kRun - 1);
    };
    const auto page_of = [&](uint32_t i) -> const uint8_t* {
        uint32_t page = 0;
        if (i < i1) {
            page = (uint32_t)p.table[b * p.table_stride + (run_of(i) >> p.page_shift)];
            if (page >= p.num_pages) {
                if (p.status && lane == 0) atomicOr(p.status, kDevBadPage);
                page = 0;
            }
        }
        return p.pages + (uint64_t)wave_uniform(page) * p.page_bytes;
    };
    const uint32_t P = 1u << p.page_shift;
    constexpr uint32_t CODE = page_code_bytes(FMT, D), STEP = page_step_bytes(FMT, D);
    // registers of a tile on its way (formats that are widened)
    constexpr int NR = FMT == kPageBf16 ? 1 : (kRun * CODE + 1023) / 1024;  // 16-byte loads of a lane
    u32x4 raw[2][NR];
    uint32_t raw_step[2];
    const auto ask = [&](uint32_t i, uint32_t buf, const uint8_t* page) {
        const uint32_t t = run_of(i), at = t & (P - 1);
        const bool whole = (t == start_of(i) + kRun * wave) & (t + kRun <= end) & ((t + kRun <= sunk) | (t >= lo));
        // the row that stands for row r of the run
        const auto row = [&](uint32_t r) {
            if (whole) return r;
            const uint32_t tok = t + r;
            if (tok >= end || t != start_of(i) + kRun * wave) return end - 1 - t;
            return tok < sunk || tok >= lo ? r : t < sunk ? sunk - 1 - t : lo - t;
        };
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const uint32_t line = ((kv ? p.H : 0) + h) * P + at;
            const uint8_t* rows = page + (uint64_t)line * CODE;
            const uint8_t* steps = page + p.steps + (uint64_t)line * STEP;
            if constexpr (FMT == kPageBf16) {
                constexpr uint32_t RPI = 1024 / CODE;  // rows of one load
                uint8_t* to = sh.kv[buf][kv] + kRun * wave * CODE;
#pragma unroll
                for (uint32_t u = 0; u < kRun / RPI; ++u) {
                    const uint32_t r = u * RPI + lane / (CODE / 16), at16 = lane % (CODE / 16);
                    // the chunk whose place is at16: places change by exclusive or, so the same change leads back
                    const uint32_t off = kv ? place_v<D>(r, at16) : place_k<D>(r, at16);
                    fetch16(rows + (off % CODE + row(r) * CODE), to + u * 1024);
                }
            } else if constexpr (FMT == kPageFp4) {
                const uint32_t r = row(lane / 4);
                if constexpr (D == 128) {
                    raw[kv][0] = *reinterpret_cast<const u32x4*>(rows + r * CODE + lane % 4 * 16);
                } else {
                    const u32x2 y = *reinterpret_cast<const u32x2*>(rows + r * CODE + lane % 4 * 8);
                    raw[kv][0] = u32x4{y.x, y.y, 0, 0};
                }
                raw_step[kv] = steps[r * STEP + lane % 4 * STEP / 4];
            } else {
#pragma unroll
                for (int u = 0; u < NR; ++u)
                    raw[kv][u] = *reinterpret_cast<const u32x4*>(rows + row((u * 1024 + lane * 16) / CODE) * CODE + lane * 16 % CODE);
                raw_step[kv] = *reinterpret_cast<const uint32_t*>(steps + row(lane % kRun) * STEP);
            }
        }
    };
    const auto put = [&](uint32_t buf) {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            uint8_t* to = sh.kv[buf][kv];
            if constexpr (FMT == kPageFp4) {
                const uint32_t r = kRun * wave + lane / 4, s = raw_step[kv] << 23;
#pragma unroll
                for (int u = 0; u < D / 32; ++u) {
                    const uint32_t y = raw[kv][0][u], chunk = lane % 4 * (D / 32) + u;
                    *reinterpret_cast<u32x4*>(to + (kv ? place_v<D>(r, chunk) : place_k<D>(r, chunk))) =
                        u32x4{widen_fp4<0>(y, s), widen_fp4<1>(y, s), widen_fp4<2>(y, s), widen_fp4<3>(y, s)};
                }
            } else if constexpr (HALF) {
#pragma unroll
                for (int u = 0; u < NR; ++u) {
                    const uint32_t r = kRun * wave + (u * 1024 + lane * 16) / D, chunk = lane * 16 % D / 8;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t a = raw[kv][u][2 * j], c = raw[kv][u][2 * j + 1];
                        u32x4 y;
                        if constexpr (FMT == kPageInt8) {
                            a ^= 0x80808080u;
                            c ^= 0x80808080u;
                            y = u32x4{widen_int8<false>(a), widen_int8<true>(a), widen_int8<false>(c), widen_int8<true>(c)};
                        } else {
                            y = u32x4{widen_fp8<false>(a), widen_fp8<true>(a), widen_fp8<false>(c), widen_fp8<true>(c)};
                        }
                        *reinterpret_cast<u32x4*>(to + (kv ? place_v<D>(r, chunk + j) : place_k<D>(r, chunk + j))) = y;
                    }
                }
                if (lane < kRun) sh.steps[buf][kv][kRun * wave + lane] = __uint_as_float(raw_step[kv]);
            }
        }
    };

    // ---- running state
    f32x16 o[CB];
#pragma unroll
    for (int n = 0; n < CB; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[n][i] = 0.0f;
    float m = kNegInf, mu = 0.0f, l = 0.0f;
    int E = -100;  // exponent taken out of the weights (HALF), which no step so far has reached
    float wmul = __builtin_amdgcn_ldexpf(1.0f, kWeightExp + 100);

    const auto tile = [&](uint32_t t0, uint32_t buf) {
        const uint8_t* kt = sh.kv[buf][0];
        const uint8_t* vt = sh.kv[buf][1];
        // whether this wave's rows see none, some or all of the tile
        if (!works || wave_hi < (int32_t)t0) return;
        const bool seen_by_window =  // all of it
            !p.window || t0 + kTokens <= p.sinks || (int32_t)t0 > wave_hi - (int32_t)p.window;
        const bool all = (int32_t)(t0 + kTokens - 1) <= wave_lo && seen_by_window;
        // whether the row sees token t0 + 4 hi + c
        const int32_t past = pos - (int32_t)t0 - 4 * (int32_t)hi;
        const int32_t left = p.window ? past - (int32_t)p.window : -0x7FFFFFFF;
        const int32_t sunk_to = p.window ? (int32_t)p.sinks - (int32_t)t0 - 4 * (int32_t)hi : 0;
        const auto counts = [&](int32_t c) { return (c <= past) & ((c > left) | (c < sunk_to)); };

        f32x16 s[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[u][i] = 0.0f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const u32x4 a = *reinterpret_cast<const u32x4*>(kt + place_k<D>(32 * u + col, 2 * k + hi));
                s[u] = mfma<FMT>(a, qf[k], s[u]);
            }
        }
        if constexpr (HALF) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f32x4 ks = *reinterpret_cast<const f32x4*>(&sh.steps[buf][0][32 * u + 8 * j + 4 * hi]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[u][4 * j + i] *= ks[i];
                }
        }
        if (!all) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    s[u][i] = counts(32 * u + 8 * (i / 4) + i % 4) ? s[u][i] : kNegInf;
        }
        float top = s[0][0];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[u][i]);
        top *= f;
        // steps of the values, brought into binary16's range by 2^-E
        float vs[HALF ? 32 : 1];
        bool move = top > m + kSlack;
        float big = 0.0f;
        if constexpr (HALF) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f32x4 y = *reinterpret_cast<const f32x4*>(&sh.steps[buf][1][32 * u + 8 * j + 4 * hi]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        vs[16 * u + 4 * j + i] = y[i];
                        big = fmaxf(big, (all | counts(32 * u + 8 * j + i)) ? y[i] : 0.0f);
                    }
                }
            move |= big >= __builtin_amdgcn_ldexpf(1.0f, E);
        }
        if (__ballot(move) != 0) {
            const auto larger = [](float a, float c) { return fmaxf(a, c); };
            const float nm = fmaxf(m, over_pair(top, larger));
            float a = nm == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m - nm);
            m = nm;
            mu = nm == kNegInf ? 0.0f : nm;
            l *= a;
            if constexpr (HALF) {
                big = over_pair(big, larger);
                const int ne = big >= __builtin_amdgcn_ldexpf(1.0f, E) ? __builtin_amdgcn_frexp_expf(big) : E;
                a *= __builtin_amdgcn_ldexpf(1.0f, E - ne);
                E = ne;
                wmul = __builtin_amdgcn_ldexpf(1.0f, kWeightExp - E);
            }
#pragma unroll
            for (int n = 0; n < CB; ++n) o[n] *= a;
        }
        u32x4 pf[4];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float e[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    e[i] = __builtin_amdgcn_exp2f(fmaf(s[u][2 * j + i], f, -mu));
                    l += e[i];
                    if constexpr (HALF) {
                        e[i] *= vs[16 * u + 2 * j + i] * wmul;
                    }
                }
                if constexpr (HALF) {
                    if (!all) {  // a step that does not count may be NaN
#pragma unroll
                        for (int i = 0; i < 2; ++i) e[i] = s[u][2 * j + i] == kNegInf ? 0.0f : e[i];
                    }
                    pf[2 * u + j / 4][j % 4] = pack_half2(e[0], e[1]);
                } else {
                    pf[2 * u + j / 4][j % 4] = pack_bf16x2(e[0], e[1]);
                }
            }
        // four tokens of one channel a read: token 4 g + (lane % 16) / 4 of the tile, channels of 64 bytes
        const uint32_t i16 = lane & 15;
        const auto values = [&](int k, int n) {
            const uint32_t chunk = 4 * n + (lane >> 4 & 1) * 2 + (i16 & 3) / 2;
            const uint32_t t = 16 * k + 4 * hi + i16 / 4;
            const auto part = [&](uint32_t token) {
                return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                     (KVC_LDS s16x4*)(vt + place_v<D>(token, chunk) + (i16 & 1) * 8)));
            };
            const u32x2 a = part(t), c = part(t + 8);
            return u32x4{a.x, a.y, c.x, c.y};
        };
        bool clean = true;
        if constexpr (!HALF) {
            if (!all) {
                // a value that is not finite, times a weight of 0, would reach rows that do not see its token
                uint32_t bad = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int n = 0; n < CB; ++n) {
                        const u32x4 y = values(k, n);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            bad |= ((y[i] & 0x7F80u) == 0x7F80u) | ((y[i] & 0x7F800000u) == 0x7F800000u);
                    }
                clean = __ballot(bad != 0) == 0;
            }
        }
        if (__builtin_expect(!clean, 0)) {
            // rows that see such a value become NaN in its channel here; below it is left out
#pragma unroll 1
            for (int t = 0; t < (int)kTokens; ++t) {
                const bool sees = counts(t - 4 * (int32_t)hi);
#pragma unroll
                for (int n = 0; n < CB; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const u32x2 y = *reinterpret_cast<const u32x2*>(vt + place_v<D>(t, 4 * n + j) + 8 * hi);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t bits = y[i / 2] >> (16 * (i % 2)) & 0x7F80u;
                            o[n][4 * j + i] = (sees & (bits == 0x7F80u)) ? __builtin_nanf("") : o[n][4 * j + i];
                        }
                    }
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int n = 0; n < CB; ++n) {
                u32x4 y = values(k, n);
                if (__builtin_expect(!clean, 0)) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        y[i] = (y[i] & 0x7F80u) == 0x7F80u ? y[i] & 0xFFFF0000u : y[i];
                        y[i] = (y[i] & 0x7F800000u) == 0x7F800000u ? y[i] & 0xFFFFu : y[i];
                    }
                }
                o[n] = mfma<FMT>(y, pf[k], o[n]);
            }
    };

    if (i0 < i1) {
        const auto arrive = [&]() {
            // LDS that other waves' loads fill is whole once each has waited for its own
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __syncthreads();
        };
        const uint8_t* page = page_of(i0);
        ask(i0, 0, page);
        page = page_of(i0 + 1);
        if (FMT != kPageBf16) put(0);
        arrive();
        for (uint32_t i = i0; i < i1; ++i) {
            const uint32_t buf = (i - i0) & 1;
            if (i + 1 < i1) {
                ask(i + 1, buf ^ 1, page);
                page = page_of(i + 2);
            }
            tile(start_of(i), buf);
            if (FMT != kPageBf16 && i + 1 < i1) put(buf ^ 1);
            arrive();
        }
    }

    // ---- output
    l = over_pair(l, [](float a, float c) { return a + c; });
    const uint64_t out_row = (uint64_t)(first + tok) * p.Hq + qh;
    if (HALF) {
        const float down = __builtin_amdgcn_ldexpf(1.0f, E - kWeightExp);
#pragma unroll
        for (int n = 0; n < CB; ++n) o[n] *= down;
    }
    if (p.splits > 1) {
        if (!has_row) return;
        const uint64_t all_rows = (uint64_t)p.rows * p.Hq;
        float* to = p.part + (split * all_rows + out_row) * D;
#pragma unroll
        for (int n = 0; n < CB; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<f32x4*>(to + 32 * n + 8 * j + 4 * hi) =
                    f32x4{o[n][4 * j], o[n][4 * j + 1], o[n][4 * j + 2], o[n][4 * j + 3]};
        if (hi == 0)
            *reinterpret_cast<float2*>(p.part + p.splits * all_rows * D + (split * all_rows + out_row) * 2) = make_float2(m, l);
        return;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    if (p.lse && has_row && hi == 0) p.lse[out_row] = (m + log2f(l)) * 0.69314718055994531f;
    // rows go through LDS, so that they are written in one piece
    constexpr uint32_t LINE = 2 * D + 16;
    static_assert(kWavesOf * 32 * LINE <= sizeof(sh.kv));
    uint8_t* mine = &sh.kv[0][0][0] + wave * 32 * LINE;
#pragma unroll
    for (int n = 0; n < CB; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<u32x2*>(mine + col * LINE + 2 * (32 * n + 8 * j + 4 * hi)) =
                u32x2{pack_bf16x2(o[n][4 * j] * inv, o[n][4 * j + 1] * inv), pack_bf16x2(o[n][4 * j + 2] * inv, o[n][4 * j + 3] * inv)};
    __builtin_amdgcn_wave_barrier();
    constexpr uint32_t LPR = 2 * D / 16;  // lanes of a row
#pragma unroll
    for (uint32_t u = 0; u < 32 * LPR / kWave; ++u) {
        const uint32_t r = u * (kWave / LPR) + lane / LPR, piece = lane % LPR;
        const uint32_t at = wave * 32 + r;
        if (at >= nrows) continue;
        const uint32_t to_tok = (row0 + at) / p.group, to_head = h * p.group + (row0 + at) % p.group;
        *reinterpret_cast<u32x4*>(p.out.data + (uint64_t)(first + to_tok) * p.out.ts + (uint64_t)to_head * p.out.hs + 8 * piece) =
            *reinterpret_cast<const u32x4*>(mine + r * LINE + 16 * piece);
    }
}

// Joins the shares of a row's tokens, a wave a row.
template <int D>
__global__ __launch_bounds__(kBlockThreads) void prompt_join_kernel(PromptParams p) {
    constexpr int C = D / kWave;
    const uint32_t lane = lane_id(), wave = wave_uniform(threadIdx.x / kWave);
    const uint64_t all_rows = (uint64_t)p.rows * p.Hq, row = (uint64_t)blockIdx.x * (kBlockThreads / kWave) + wave;
    if (row >= all_rows) return;
    const int32_t n = (int32_t)(row / p.Hq);
    if (n < p.starts[0] || n >= p.starts[p.n]) return;
    const float* ml = p.part + p.splits * all_rows * D;
    float M = kNegInf;
    for (uint32_t s = 0; s < p.splits; ++s) M = fmaxf(M, ml[(s * all_rows + row) * 2]);
    const float mu = M == kNegInf ? 0.0f : M;
    float total = 0.0f, y[C] = {};
    for (uint32_t s = 0; s < p.splits; ++s) {
        const float2 x = *reinterpret_cast<const float2*>(ml + (s * all_rows + row) * 2);
        const float a = __builtin_amdgcn_exp2f(x.x - mu);
        total = fmaf(x.y, a, total);
#pragma unroll
        for (int c = 0; c < C; ++c) y[c] += p.part[(s * all_rows + row) * D + C * lane + c] * a;
    }
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    uint16_t* to = p.out.data + (uint64_t)n * p.out.ts + (row % p.Hq) * p.out.hs + C * lane;
    if constexpr (C == 2)
        *reinterpret_cast<uint32_t*>(to) = pack_bf16x2(y[0] * inv, y[1] * inv);
    else
        *to = (uint16_t)pack_bf16x2(y[0] * inv, 0.0f);
    if (p.lse && lane == 0) p.lse[row] = (M + log2f(total)) * 0.69314718055994531f;
}

template <int FMT, int D>
hipError_t launch(const PromptParams& p, uint32_t grid, hipStream_t stream) {
    return launch_kernel(prompt_kernel<FMT, D>, dim3(grid), dim3(kWavesOf * kWave), stream, p);
}
template <int D>
hipError_t launch_of(uint32_t format, const PromptParams& p, uint32_t grid, hipStream_t stream) {
    switch (format) {
        case kPageBf16: return launch<kPageBf16, D>(p, grid, stream);
        case kPageInt8: return launch<kPageInt8, D>(p, grid, stream);
        case kPageFp8: return launch<kPageFp8, D>(p, grid, stream);
        default: return launch<kPageFp4, D>(p, grid, stream);
    }
}

// Workgroups that the GPU holds at once, and the fewest tokens of a share.
constexpr uint64_t kPlaces = 512, kMinShare = 256;

}  // namespace

PromptPlan prompt_plan(uint32_t n_seqs, uint32_t n_tokens, uint32_t H, uint32_t Hq, uint32_t d, uint64_t max_tokens,
                       uint32_t window, uint32_t sinks) {
    PromptPlan a{kRows, 1, 0, 256, 256};
    const uint64_t group = Hq / H;
    a.blocks = n_tokens * group / kRows + n_seqs;
    // with a window, a block's rows see the tokens of one row and as many more as the block has tokens
    const uint64_t seen = window ? seen_tokens(max_tokens, (uint64_t)window + kRows / group, sinks) : max_tokens;
    const uint64_t most = (seen + kMinShare - 1) / kMinShare;
    const uint64_t shares = a.blocks ? kPlaces / (H * a.blocks) : 1;
    a.splits = (uint32_t)(shares < 1 || most < 1 ? 1 : shares < most ? shares : most);
    const uint64_t rows = (uint64_t)n_tokens * Hq, each = (uint64_t)(d + 2) * 4;
    if (a.splits > 1) a.bytes = align_up(a.splits * rows * each, 256);
    if (most > 1) {
        // at most kPlaces shares of kRows rows
        const uint64_t bound = rows * most < kPlaces * kRows ? rows * most : kPlaces * kRows;
        a.room = align_up(bound * each, 256);
        if (a.room < 256) a.room = 256;
    }
    return a;
}

hipError_t launch_attend_prompt(const PromptArgs& a, const PromptPlan& plan, hipStream_t stream) {
    PromptParams p{};
    const PageLayout& lay = a.tail.lay;
    p.q = a.q;
    p.out = a.out;
    p.lse = a.lse;
    p.status = a.status;
    p.starts = a.starts;
    p.lens = a.tail.lens;
    p.table = a.tail.table;
    p.pages = a.tail.pages;
    p.table_stride = a.tail.table_stride;
    p.page_bytes = lay.page_bytes;
    p.steps = lay.steps;
    p.n = a.n;
    p.rows = a.rows;
    p.H = a.H;
    p.Hq = a.Hq;
    p.group = a.Hq / a.H;
    p.table_cols = a.tail.table_cols;
    p.num_pages = lay.num_pages;
    p.page_shift = 31 - __builtin_clz(lay.P);
    p.window = a.tail.window;
    p.sinks = a.tail.sinks;
    p.splits = plan.splits;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.part = static_cast<float*>(a.ws);
    const uint32_t grid = (uint32_t)(plan.blocks * a.H * plan.splits);
    const hipError_t e = a.d == 64 ? launch_of<64>(lay.format, p, grid, stream) : launch_of<128>(lay.format, p, grid, stream);
    if (e != hipSuccess || plan.splits == 1) return e;
    const uint64_t rows = (uint64_t)a.rows * a.Hq;
    return launch_kernel(a.d == 64 ? prompt_join_kernel<64> : prompt_join_kernel<128>,
                         dim3((uint32_t)((rows + 3) / 4)), dim3(kBlockThreads), stream, p);
}

}  // namespace kvc
