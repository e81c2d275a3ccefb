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
// Bound: pages, memory; the codes are read once, and a tile costs d / 4 matrix
// instructions per 16 rows, far below their rate (32 sequences of up to 16384
// tokens, 8 kv heads of 128, e4m3: 98 us, 5.6 TB/s of codes and steps). A pool
// holds 178 bytes for a token's key and value of 128 channels instead of 264, and
// many rows share them: there the vector instructions of widening and softmax
// and the matrix instructions, which a SIMD issues one at a time, bound it
// (131071 tokens, 8 kv heads of 128, 60 rows: 77 us, 2.4 TB/s; of a SIMD's
// cycles the VALU takes 72 %, the matrix core 18 %). Short calls are bound by latency: three
// dependent reads, a tile, the join of four waves: 5.5 us.
//
// Tried and left out: keeping two tiles of loads in registers (spills, or the same
// time); sharing widened tokens among the waves through LDS (a quarter fewer
// vector instructions, the same time); joining parts in the workgroup that ends a
// unit (the agent-scope fences write back and drop L2: 20 -> 78 us).
//
// Number formats: int8 and e4m3 codes, and the pool's levels, are widened to
// binary16, where codes are exact (levels: within 2^-17.5, see kLevelFactor). Queries go to
// binary16 after division by a power of two per row (the row's largest
// becomes 2^14..2^15, so what is lost is below 2^-39 of it). Weights p * step
// go to binary16 (2^-12) after division by 2^E, E the wave's largest step
// exponent so far, times 2^12: the largest stays below 2^16 (m may lag the
// true maximum by kSlack), and weights down to 2^-26 of it keep all bits. A
// bf16 cache uses bf16 instructions, each p split into two bf16 terms, since
// one alone (2^-9) would show next to the output's own rounding.
//
// m is moved only when a tile's maximum passes it by kSlack (exponents of 2):
// most tiles then need no exchange between lanes and no rescaling. Logits are
// rounded products of K q with the row's factor, so the maximum's difference to m
// is exact however large they are: a fused product * factor - m leaves the rounding
// of m, which passes binary16's range at logits of 2^25 (and costs the same: the
// compiler makes matrix results canonical before it compares them).
#include "attend.h"
#include "codebook.h"
#include "kernels_common.h"

#include <type_traits>

namespace kvc {
namespace {

constexpr int kDevBadHeader = 1, kDevBadPage = 32, kDevBadLength = 64;  // KVC_DEV_*
constexpr int kFmtBf16 = 0, kFmtInt8 = 1, kFmtFp8 = 2, kFmtPool = 3;
constexpr int kWaves = 4;
constexpr uint32_t kTile = 32;
constexpr uint32_t kBlock = kWaves * kTile;  // tokens of one step of a workgroup
constexpr uint32_t kPageRun = 32 * kBlock;   // 32 tiles a wave: a page number for 16 tokens in each of 64 lanes
constexpr float kSlack = 3.0f;
constexpr int kWeightExp = 12;
constexpr int kMinExp = -100;  // steps below 2^-100 are taken with this exponent
constexpr float kNegInf = -__builtin_inff();

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t ushort2_t __attribute__((ext_vector_type(2)));

struct Common {
    RowsDev q, out;
    float* lse;
    int32_t* status;
    uint32_t n, H, Hq, group;  // sequences (or agents), kv heads, query heads, Hq / H
    uint32_t direct;           // one source: what needs no joining is written as output
    float scale_log2;
};

// One source of tokens: a pool's layer, or pages. Its units are (sequence, kv
// head, row block), the pool's (kv head, row block); a unit's tokens come
// in blocks of kBlock. Workgroup w of W takes an equal share of all blocks in
// unit order; with `whole`, workgroup w is unit w.
struct Source {
    uint32_t rows, row_blocks, W, whole;
    // partial results: slots of 16 RT rows x (d sums, then {m, l}). The part of a unit that workgroup w starts is
    // slot 2w + 1, one that it continues slot 2w; whole units (where they are joined at all) come behind, at 2W
    // (at 0 with `whole`).
    float* part;
    uint2* info;  // of each unit: first slot, number of parts (0: written as output)
    // pool
    const uint8_t* pool;
    PoolLayout lay;
    uint32_t L, T, layer;
    uint32_t more;  // shares of `each` blocks, the first `more` of them one larger
    uint64_t each;
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
// levels first .. first + 3. As they are the levels would lose up to 0.83 of 2^-12,
// every token alike, so no sum over tokens averages it out; times this factor, which the
// transform takes out again, each lies within 0.0212 of 2^-12 of a binary16 number.
constexpr double kLevelFactor = 1.8587914;
constexpr uint32_t level_half(int i) {
    const float pos[4] = {kLv0, kLv1, kLv2, kLv3};
    return __builtin_bit_cast(uint16_t, (_Float16)(float)((i < 4 ? -pos[3 - i] : pos[i - 4]) * kLevelFactor));
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
    uint32_t v[2][3];  // one word of each plane of one token per run of 16 (see gather_bytes)
    uint2 vs[2];       // four binary16 sizes per run
};

// a where the mask has ones, b elsewhere; one instruction, which the compiler
// would take apart again for the bits that are used in the end.
__device__ __forceinline__ uint32_t merge(uint32_t mask, uint32_t a, uint32_t b) {
    uint32_t r = (a & mask) | (b & ~mask);
    asm("" : "+v"(r));
    return r;
}

// Bytes of four tokens, from four lanes that each hold a word of one: lane
// 4 b + w of 16 gets byte b of word w of tokens 0..3, whose words are in
// lanes w, 4 + w, 8 + w, 12 + w. Rotations by 4, 8 and 12 lanes bring the words
// of tokens b - 1, b - 2 and b - 3 (mod 4); the selectors, which depend on b,
// place one byte of each.
__device__ __forceinline__ void gather_selectors(uint32_t b, uint32_t& sel_a, uint32_t& sel_b) {
    const auto at = [](uint32_t token, uint32_t byte) { return (byte ^ 0x0Cu) << (8 * (token & 3)); };
    sel_a = 0x0C0C0C0Cu ^ at(b, b) ^ at(b - 1, 4 + b);
    sel_b = 0x0C0C0C0Cu ^ at(b - 2, b) ^ at(b - 3, 4 + b);
}
__device__ __forceinline__ uint32_t gather_bytes(uint32_t own, uint32_t sel_a, uint32_t sel_b) {
    const uint32_t r4 = (uint32_t)__builtin_amdgcn_mov_dpp((int)own, 0x124, 0xF, 0xF, true);
    const uint32_t r8 = (uint32_t)__builtin_amdgcn_mov_dpp((int)own, 0x128, 0xF, 0xF, true);
    const uint32_t r12 = (uint32_t)__builtin_amdgcn_mov_dpp((int)own, 0x12C, 0xF, 0xF, true);
    return __builtin_amdgcn_perm(r4, own, sel_a) | __builtin_amdgcn_perm(r12, r8, sel_b);
}

// First channel of matrix row 4 g + r of the value products.
template <int FMT, int D>
__device__ __forceinline__ uint32_t channel_of(uint32_t g, uint32_t r) {
    if (FMT != kFmtPool) return (4 * g + r) * (D / 16);
    // lane 4 g + r holds byte g of word r (d = 128), or a nibble of it
    return D == 128 ? 32 * r + 8 * g : 32 * (r & 1) + 8 * g + 4 * (r >> 1);
}

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

// What no workgroup of a launch writes, at an address that is the same in all
// lanes: read through the scalar cache, without a wait until it is used.
template <class T>
__device__ __forceinline__ T scalar_load(const void* a) {
    return *(const __attribute__((address_space(4))) T*)(uint64_t)a;
}

// (all words at once: compared one after another, each would wait for its load)
__device__ __forceinline__ bool pool_header_ok(const Source& p, uint32_t H, uint32_t D) {
    const u32x4 a = scalar_load<u32x4>(p.pool), b = scalar_load<u32x4>(p.pool + 16), c = scalar_load<u32x4>(p.pool + 48);
    const uint64_t t = (uint64_t)c.z | ((uint64_t)c.w << 32);
    return (a.x == kPoolMagic) & (a.y == (1u | (1u << 16))) & (a.z == p.L) & (a.w == H) & (b.x == p.T) & (b.y == D) &
           (t == p.lay.total);
}

// A sequence's length, within what its table's row holds.
__device__ __forceinline__ uint32_t clamp_length(const Source& p, int32_t len) {
    const uint32_t most = p.table_cols << p.page_shift;
    return len < 0 ? 0 : (uint32_t)len > most ? most : (uint32_t)len;
}
__device__ __forceinline__ bool bad_length(const Source& p, int32_t len) {
    return len < 0 || (uint32_t)len > p.table_cols << p.page_shift;
}
// Blocks of a length; an empty sequence has one, without tokens.
__device__ __forceinline__ uint32_t blocks_of(uint32_t len) { return len <= kBlock ? 1 : (len + kBlock - 1) / kBlock; }

// Query row r (of the unit's rows) -> sequence and query head.
template <int FMT>
__device__ __forceinline__ void row_of(const Common& p, uint32_t b, uint32_t h, uint32_t r, uint32_t& seq,
                                       uint32_t& qh) {
    if (FMT == kFmtPool) {
        seq = r / p.group;
        qh = h * p.group + r % p.group;
    } else {
        seq = b;
        qh = h * p.group + r;
    }
}

template <int CTRL>
__device__ __forceinline__ float dpp_move(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
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
    // partners lane ^ 1, 2, 4, 8 by DPP: quad permutes, a mirror of 8 and then of
    // 4, a rotation by 8 of 16
    const auto step = [&](int h, auto partner) {
        const float s = (lane & h) ? -1.0f : 1.0f;
#pragma unroll
        for (int i = 0; i < C; ++i) y[i] = fmaf(s, y[i], partner(y[i]));
    };
    step(1, [](float v) { return dpp_xor1(v); });
    step(2, [](float v) { return dpp_xor2(v); });
    step(4, [](float v) { return dpp_move<0x1B>(dpp_move<0x141>(v)); });
    step(8, [](float v) { return dpp_move<0x128>(v); });
}

// Waves of a SIMD, which sets the register budget (512 / waves) and how many
// workgroups a CU holds.
constexpr int waves_per_simd(int d, int rt) { return d == 64 ? (rt == 1 ? 3 : 2) : 2; }

// LDS of a workgroup. (Without its alignment, accesses of four floats come out in pairs.)
template <int D, int RT>
struct Shared {
    alignas(16) float ml[kWaves][RT * 16][2];
    alignas(16) float os[RT][kWaves][16][D + 4];
    uint32_t sums[kWaves];
    uint32_t found[3];  // sequence, blocks before it, its blocks
};

// Over the four lanes that hold a query row (lane % 16), in all of them: rows of 16
// lanes change places, then halves.
template <class T, class F>
__device__ __forceinline__ T over_groups(T v, F join) {
    const uint32_t a = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    const uint32_t b = __builtin_bit_cast(uint32_t, join(__builtin_bit_cast(T, (uint32_t)r[0]), __builtin_bit_cast(T, (uint32_t)r[1])));
    const auto h = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return join(__builtin_bit_cast(T, (uint32_t)h[0]), __builtin_bit_cast(T, (uint32_t)h[1]));
}

// Over the wave's lanes up to this one, by moves inside rows of 16 and the last
// lanes of rows to the rows behind them (with LDS permutes: some 100 cycles a step).
template <class T, class F>
__device__ __forceinline__ T scan_wave(T v, T none, F join) {
    const auto step = [&](auto ctrl, auto rows) {
        const int o = __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none), __builtin_bit_cast(int, v),
                                                  decltype(ctrl)::value, decltype(rows)::value, 0xF, false);
        v = join(v, __builtin_bit_cast(T, o));
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
__device__ __forceinline__ uint32_t scan_lanes(uint32_t v) {
    return scan_wave(v, 0u, [](uint32_t a, uint32_t b) { return a + b; });
}
__device__ __forceinline__ float last_lane(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// Sum over the workgroup's threads before this one, and the sum of all.
__device__ __forceinline__ uint32_t scan_threads(uint32_t v, uint32_t* sums, uint32_t& all) {
    const uint32_t lane = lane_id(), wave = threadIdx.x / kWave;
    const uint32_t s = scan_lanes(v);
    if (lane == 63) sums[wave] = s;
    __syncthreads();
    uint32_t before = 0;
    all = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        if ((uint32_t)i < wave) before += sums[i];
        all += sums[i];
    }
    return before + s - v;
}

// The share of workgroup w.
template <int FMT, int D, int RT>
__device__ __forceinline__ void attend_share(const Common& p, const Source& src, uint32_t w, Shared<D, RT>& sh) {
    constexpr int KS = D / 32;   // key product steps
    constexpr int NC = D / 16;   // channels of a lane, value products
    constexpr bool HALF = FMT != kFmtBf16;
    using R = Raw<FMT, D>;
    const uint32_t lane = lane_id(), c = lane & 15, g = lane >> 4;
    const uint32_t wave = wave_uniform(threadIdx.x / kWave);
    const uint32_t per_seq = p.H * src.row_blocks;  // units of a sequence

    // ---- this workgroup's blocks: `left` of them, from block `off` of unit (b, hr)
    uint32_t b = 0, hr = 0, off = 0;
    // shares of `each` blocks, the first `more` of them one larger; this one begins at x0
    uint64_t each = 0, x0 = 0, left;
    uint32_t more = 0;
    const auto begin_share = [&]() {
        x0 = each * w + (w < more ? w : more);
        left = each + (w < more);
    };
    const auto share = [&](uint64_t total) {
        // no empty shares
        if (w >= total) return false;
        const uint32_t W = total < src.W ? (uint32_t)total : src.W;
        if (w >= W) return false;
        divmod_u64(total, W, each, more);
        begin_share();
        return true;
    };
    if (FMT == kFmtPool) {
        const uint32_t nb = blocks_of(src.T);
        if (src.whole) {
            hr = w;
            left = nb;
        } else {
            each = src.each;
            more = src.more;
            begin_share();
            uint64_t q;
            divmod_u64(x0, nb, q, off);
            hr = (uint32_t)q;
        }
    } else if (src.whole) {
        b = w / per_seq;
        hr = w % per_seq;
        left = 1u << 31;
    } else {
        // the sequence that holds block x0, the blocks before it and its own
        uint32_t before, mine;
        uint64_t q64;
        uint32_t part;
        if (p.n <= kWave) {
            // a sequence a lane, in every wave for itself
            const uint32_t v = lane < p.n ? blocks_of(clamp_length(src, src.lens[lane])) : 0;
            const uint32_t up = scan_lanes(v);
            if (!share((uint64_t)__builtin_amdgcn_readlane(up, 63) * per_seq)) return;
            divmod_u64(x0, per_seq, q64, part);
            b = __builtin_popcountll(__ballot(up <= (uint32_t)q64));  // sequences that end before
            mine = __builtin_amdgcn_readlane(v, b & 63);
            before = __builtin_amdgcn_readlane(up, b & 63) - mine;
        } else {
            // every thread counts a run of sequences; the one whose run holds the block then finds it
            const uint32_t run = (p.n + kWaves * kWave - 1) / (kWaves * kWave);
            const uint32_t s0 = threadIdx.x * run, s1 = s0 + run < p.n ? s0 + run : p.n;
            uint32_t v = 0, all;
            for (uint32_t s = s0; s < s1; ++s) v += blocks_of(clamp_length(src, src.lens[s]));
            const uint32_t at0 = scan_threads(v, sh.sums, all);
            if (!share((uint64_t)wave_uniform(all) * per_seq)) return;
            divmod_u64(x0, per_seq, q64, part);
            const uint32_t q = (uint32_t)q64;
            if (q >= at0 && q - at0 < v) {
                uint32_t at = at0, s = s0, nb = 0;
                for (; s < s1; ++s) {
                    nb = blocks_of(clamp_length(src, src.lens[s]));
                    if (q - at < nb) break;
                    at += nb;
                }
                sh.found[0] = s;
                sh.found[1] = at;
                sh.found[2] = nb;
            }
            __syncthreads();
            b = wave_uniform(sh.found[0]);
            before = wave_uniform(sh.found[1]);
            mine = wave_uniform(sh.found[2]);
        }
        divmod_u64(x0 - (uint64_t)before * per_seq, mine, q64, off);
        hr = (uint32_t)q64;
    }

    uint64_t first = x0 - off;  // the unit's first block
    for (uint32_t nb = 0; left != 0; off = 0, ++hr, first += nb) {
        if (FMT != kFmtPool && hr == per_seq) {
            hr = 0;
            ++b;
        }
        if (FMT == kFmtPool ? hr >= per_seq : b >= p.n) break;
        const uint32_t h = hr / src.row_blocks, rb = hr % src.row_blocks;

        // everything that can be asked for at once: the queries (row 16 rt + c,
        // channels as the key loads have them), the length, the first page numbers
        uint32_t qw[RT][KS][4];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const uint32_t r = (rb * RT + rt) * 16 + c;
            uint32_t seq, qh;
            row_of<FMT>(p, b, h, r < src.rows ? r : 0, seq, qh);
            const uint8_t* qp = reinterpret_cast<const uint8_t*>(p.q.data + (uint64_t)seq * p.q.ts + (uint64_t)qh * p.q.hs);
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const uint32_t ch = HALF ? (s / 2) * 64 + g * 16 + (s % 2) * 8 : s * 32 + g * 8;
                load_words(qp + 2 * ch, qw[rt][s]);
            }
        }
        // page numbers of this wave's 16-token runs: run i of tile t in lane 2t + i
        // (whole rows of the table can be read, whatever the length)
        const uint32_t run0 = ((lane >> 1) * kWaves + wave) * kTile + (lane & 1) * 16;
        const auto load_pages = [&](uint32_t base) {
            const uint32_t t = (base + run0) >> src.page_shift;
            return src.table[b * src.table_stride + (t < src.table_cols ? t : 0)];
        };
        int32_t given = 0, page = 0;
        if (FMT != kFmtPool) {
            given = src.lens[b];
            page = load_pages(off * kBlock);
        }
        const uint32_t len = FMT == kFmtPool ? src.T : wave_uniform(clamp_length(src, given));
        if (FMT != kFmtPool && hr == 0 && off == 0 && threadIdx.x == 0 && bad_length(src, given) && p.status)
            atomicOr(p.status, kDevBadLength);
        nb = blocks_of(len);
        const uint32_t take = nb - off < left ? nb - off : (uint32_t)left;
        left -= take;
        if (FMT != kFmtPool && src.whole) left = 0;
        const uint32_t begin = off * kBlock;
        const uint32_t end = off + take == nb ? len : begin + take * kBlock;

        const uint64_t vec0 = FMT == kFmtPool ? ((uint64_t)src.layer * p.H + h) * src.T : 0;  // the head's first vector
        uint32_t my_page = 0;
        const auto take_pages = [&](uint32_t base) {
            const bool counts = base + run0 < end, ok = (uint32_t)page < src.num_pages;
            if (counts && !ok && p.status) atomicOr(p.status, kDevBadPage);
            my_page = counts && ok ? (uint32_t)page : 0;
        };
        if (FMT != kFmtPool) take_pages(begin);
        const auto load = [&](uint32_t t0, uint32_t it, R& x) {
            if constexpr (FMT == kFmtPool) {
                const uint64_t vec = vec0 + t0;
                const uint32_t last = src.T - t0 - 1;  // tokens behind the last are the last again (masked below)
                const uint8_t* kb = src.pool + src.lay.k_codes + vec * D;
                const uint8_t* vb = src.pool + src.lay.v_codes + vec * (3 * D / 8);
                const uint8_t* sb = src.pool + src.lay.v_scale + vec * 2;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t t = 16 * i + c < last ? 16 * i + c : last;
#pragma unroll
                    for (int s = 0; s < D / 64; ++s)
                        x.k[i][s] = *reinterpret_cast<const uint4*>(kb + t * D + 64 * s + 16 * g);
                }
                const uint32_t word = 4 * (D == 128 ? c & 3 : c & 1);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t t1 = 16 * i + 4 * g + (c >> 2), t = t1 < last ? t1 : last;
#pragma unroll
                    for (int q = 0; q < 3; ++q)
                        x.v[i][q] = *reinterpret_cast<const uint32_t*>(vb + t * (3 * D / 8) + q * (D / 8) + word);
                    // sizes of four tokens; behind the last token, its own again (masked below)
                    const uint32_t s1 = 16 * i + 4 * g;
                    if (s1 + 3 <= last) {
                        __builtin_memcpy(&x.vs[i], sb + 2 * s1, 8);
                    } else {
                        uint32_t z[4];
#pragma unroll
                        for (uint32_t j = 0; j < 4; ++j)
                            z[j] = *reinterpret_cast<const uint16_t*>(sb + 2 * (s1 + j < last ? s1 + j : last));
                        x.vs[i] = make_uint2(z[0] | z[1] << 16, z[2] | z[3] << 16);
                    }
                }
            } else {
                constexpr uint32_t ROW = FMT == kFmtBf16 ? 2 * D : D;
                const uint32_t P = 1u << src.page_shift;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t pg = __builtin_amdgcn_readlane(my_page, (2 * it + i) & 63);
                    const uint8_t* pb = src.pages + (uint64_t)pg * src.page_bytes;
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
                        const float4 a = *reinterpret_cast<const float4*>(pb + src.steps + (uint64_t)(kl + 4 * g) * 4);
                        const float4 w = *reinterpret_cast<const float4*>(pb + src.steps + (uint64_t)(vl + 4 * g) * 4);
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
        R x;
        if (begin + wave * kTile < end) load(begin + wave * kTile, 0, x);
        // looked at before anything is written: the loads do not depend on it
        const bool header = FMT != kFmtPool || pool_header_ok(src, p.H, D);

        u32x4 qf[RT][KS];
        float qscale[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const uint32_t(&z)[KS][4] = qw[rt];
            // a row that is none is a zero; the factor of a row's logits is kept
            // >= 0, so that the largest product is the largest logit: a negative
            // scale turns the queries' signs
            const bool live = (rb * RT + rt) * 16 + c < src.rows;
            qscale[rt] = fabsf(p.scale_log2);
            if (HALF) {
                ushort2_t top = 0;
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        top = __builtin_elementwise_max(top, __builtin_bit_cast(ushort2_t, z[s][i] & 0x7FFF7FFFu));
                uint32_t big = top.x > top.y ? top.x : top.y;
                big = over_groups(big, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
                // largest magnitude to [2^14, 2^15), by 2^112 at most, which brings the smallest
                // bf16 into range; Inf and NaN stay what they are
                int e = (big == 0 || big >= 0x7F80u) ? 0 : 15 - __builtin_amdgcn_frexp_expf(__uint_as_float(big << 16));
                e = e < 112 ? e : 112;
                const float f = live ? copysignf(__builtin_amdgcn_ldexpf(1.0f, e), p.scale_log2) : 0.0f;
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int i = 0; i < 4; ++i) qf[rt][s][i] = pack_half2(bf16_lo(z[s][i]) * f, bf16_hi(z[s][i]) * f);
                qscale[rt] = __builtin_amdgcn_ldexpf(qscale[rt], -e);
            } else {
                const uint32_t turn = p.scale_log2 < 0.0f ? 0x80008000u : 0;
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int i = 0; i < 4; ++i) qf[rt][s][i] = live ? z[s][i] ^ turn : 0;
            }
        }
        // A logit is a sum of codes (below 2^31) times its row's factor and its key's step, either of which
        // may lie near an end of binary32's range. A factor up to 1 comes first: that sum cannot
        // overflow. One above 1 (queries from 2^18 on) comes last, so that nothing overflows before the logit does.
        bool above = false;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) above |= qscale[rt] > 1.0f;
        const bool late = HALF && __ballot(above) != 0;
        float step = 0.0f;
        if (FMT == kFmtPool) {
            step = reinterpret_cast<const float*>(src.pool + src.lay.k_scale)[src.layer];
            if (!late) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) qscale[rt] *= step;
            }
        }

        // running state
        f32x4 o[RT][NC];
        float m[RT], mu[RT], l[RT];
        int E = kMinExp;  // exponent taken out of the weights (HALF)
        float elimit = __builtin_amdgcn_ldexpf(1.0f, kMinExp);  // 2^E, which no step so far has reached
        float wmul = __builtin_amdgcn_ldexpf(1.0f, kWeightExp - kMinExp);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            m[rt] = kNegInf;
            mu[rt] = 0.0f;
            l[rt] = 0.0f;
#pragma unroll
            for (int n = 0; n < NC; ++n) o[rt][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }

        uint32_t sel_a = 0, sel_b = 0;
        if (FMT == kFmtPool) gather_selectors(c >> 2, sel_a, sel_b);

        // One tile: its loads are in x; those of the next one (at t_next, if
        // below end) go out as soon as x has been widened. PART: the tile ends
        // behind `end`.
        const auto tile = [&](auto part, uint32_t t0, uint32_t t_next, uint32_t it, R& x) {
            constexpr bool PART = decltype(part)::value;
            const uint32_t live = end - t0;
            f32x4 s[RT][2];
            {
                u32x4 kf[2][KS];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        if (HALF) {
                            const uint4& y = x.k[i][k / 2];
                            uint32_t a = k % 2 ? y.z : y.x, d = k % 2 ? y.w : y.y;
                            if (FMT != kFmtFp8) {
                                a ^= 0x80808080u;
                                d ^= 0x80808080u;
                            }
                            constexpr int F = FMT == kFmtFp8 ? kFmtFp8 : kFmtInt8;
                            kf[i][k] = u32x4{widen<F, false>(a), widen<F, true>(a), widen<F, false>(d), widen<F, true>(d)};
                        } else {
                            const uint4& y = x.k[i][k];
                            kf[i][k] = u32x4{y.x, y.y, y.z, y.w};
                        }
                    }
                }
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        s[rt][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int k = 0; k < KS; ++k) s[rt][i] = mfma<FMT>(kf[i][k], qf[rt][k], s[rt][i]);
                    }
            }
            // value operands: token pairs of one channel
            u32x4 vf[NC];
            float vs[8], ks[8];
            if constexpr (FMT == kFmtPool) {
                constexpr uint32_t l0 = level_bytes(0, 0), l1 = level_bytes(4, 0);
                constexpr uint32_t h0 = level_bytes(0, 8), h1 = level_bytes(4, 8);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t pl[3];  // byte j: the lane's byte of the plane of token j
#pragma unroll
                    for (int q = 0; q < 3; ++q) {
                        pl[q] = gather_bytes(x.v[i][q], sel_a, sel_b);
                        if (D == 64) pl[q] >>= (c >> 1 & 1) * 4;  // its nibble: what comes in above is not used
                    }
                    // bits of two planes next to one another, for even and odd channels
                    const uint32_t even = merge(0x55555555u, pl[0], pl[1] << 1), odd = merge(0x55555555u, pl[0] >> 1, pl[1]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // the codes of channels k and k + 4: the low three bits of each nibble
                        const uint32_t two = k % 2 ? odd : even;
                        const uint32_t code = merge(0x33333333u, k < 2 ? two : two >> 2,
                                                    k < 2 ? pl[2] << (k < 2 ? 2 - k : 0) : pl[2] >> (k < 2 ? 0 : k - 2));
#pragma unroll
                        for (int n = k; n < NC; n += 4) {
                            const uint32_t sel = (n == k ? code : code >> 4) & 0x07070707u;
                            const uint32_t lo = __builtin_amdgcn_perm(l1, l0, sel), hi = __builtin_amdgcn_perm(h1, h0, sel);
                            vf[n][2 * i] = __builtin_amdgcn_perm(hi, lo, 0x05010400u);
                            vf[n][2 * i + 1] = __builtin_amdgcn_perm(hi, lo, 0x07030602u);
                        }
                    }
                    const uint32_t w[2] = {x.vs[i].x, x.vs[i].y};
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const half2_t s2 = __builtin_bit_cast(half2_t, w[j]);
                        vs[4 * i + 2 * j] = (float)s2.x;
                        vs[4 * i + 2 * j + 1] = (float)s2.y;
                    }
                }
            } else {
                if (PART) {
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
                if constexpr (FMT != kFmtBf16) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        vs[j] = x.vs[j];
                        ks[j] = x.ks[j];
                    }
                }
            }
            if (t_next < end) load(t_next, it + 1, x);

            // logits (in powers of two), their maxima, and the steps' largest
            float y[RT][8], top[RT];
            bool move = false;
            if (__builtin_expect(late, 0)) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float k = FMT == kFmtPool ? step : ks[j];
                        const bool last = qscale[rt] > 1.0f;
                        y[rt][j] = s[rt][j >> 2][j & 3] * (last ? k : qscale[rt]) * (last ? qscale[rt] : k);
                    }
            } else {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        y[rt][j] = s[rt][j >> 2][j & 3] * qscale[rt];
                        if constexpr (FMT == kFmtInt8 || FMT == kFmtFp8) y[rt][j] *= ks[j];
                    }
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (PART) y[rt][j] = (j < 4 ? 0 : 16) + 4 * g + (j & 3) < live ? y[rt][j] : kNegInf;
                }
                top[rt] = y[rt][0];
#pragma unroll
                for (int j = 1; j < 8; ++j) top[rt] = fmaxf(top[rt], y[rt][j]);
                move |= top[rt] > m[rt] + kSlack;
            }
            float big = 0.0f;
            if (HALF) {
#pragma unroll
                for (int j = 0; j < 8; ++j) big = fmaxf(big, vs[j]);
                move |= big >= elimit;
            }
            if (__ballot(move) != 0) {
                const auto larger = [](float a, float b) { return fmaxf(a, b); };
                float shrink = 1.0f;
                if (HALF) {
                    big = over_groups(big, larger);
                    const int e = __builtin_amdgcn_frexp_expf(big), ne = big >= elimit ? e : E;
                    shrink = __builtin_amdgcn_ldexpf(1.0f, E - ne);
                    E = ne;
                    elimit = __builtin_amdgcn_ldexpf(1.0f, E);
                    wmul = __builtin_amdgcn_ldexpf(1.0f, kWeightExp - E);
                }
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const float nm = fmaxf(m[rt], over_groups(top[rt], larger));
                    const float a = nm == kNegInf ? 1.0f : exp2_fast(m[rt] - nm);
                    m[rt] = nm;
                    mu[rt] = nm == kNegInf ? 0.0f : nm;
                    l[rt] *= a;
#pragma unroll
                    for (int n = 0; n < NC; ++n) o[rt][n] *= a * shrink;
                }
            }
            if (HALF) {
#pragma unroll
                for (int j = 0; j < 8; ++j) vs[j] *= wmul;
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                float w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float e = exp2_fast(y[rt][j] - mu[rt]);
                    // by the token, not by its logit: -inf * 0 has no sign
                    if (PART) e = (j < 4 ? 0 : 16) + 4 * g + (j & 3) < live ? e : 0.0f;
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
                    for (int n = 0; n < NC; ++n) o[rt][n] = mfma_bf16(vf[n], hi, o[rt][n]);
#pragma unroll
                    for (int n = 0; n < NC; ++n) o[rt][n] = mfma_bf16(vf[n], lo, o[rt][n]);
                }
            }
        };

        for (uint32_t base = begin; base < end; base += kPageRun) {
            if (base != begin) {  // the next page numbers (the pool needs none: one round)
                page = load_pages(base);
                take_pages(base);
                if (base + wave * kTile < end) load(base + wave * kTile, 0, x);
            }
            const uint32_t stop = FMT == kFmtPool || end - base <= kPageRun ? end : base + kPageRun;
            uint32_t it = 0, t0 = base + wave * kTile;
            for (; t0 + kTile <= stop; t0 += kBlock, ++it)
                tile(std::false_type{}, t0, t0 + kBlock < stop ? t0 + kBlock : end, it, x);
            if (t0 < stop) tile(std::true_type{}, t0, end, it, x);
            if (FMT == kFmtPool) break;
        }
        if (FMT == kFmtPool && !header) {
            if (threadIdx.x == 0 && p.status) atomicOr(p.status, kDevBadHeader);
            return;
        }

        // ---- join the waves: m and l first, then the sums
        const bool whole = take == nb;
        const uint32_t slot = whole ? (src.whole ? 0 : 2 * src.W) + b * per_seq + hr : off ? 2 * w : 2 * w + 1;
        if (off == 0 && threadIdx.x == 0 && !(src.whole && p.direct)) {
            // parts: up to the workgroup whose share has the unit's last block
            uint32_t parts = p.direct ? 0 : 1;
            if (!whole) {
                const uint64_t last = first + nb - 1, large = (each + 1) * more;
                uint64_t at;
                uint32_t rest;
                if (last < large)
                    divmod_u64(last, (uint32_t)each + 1, at, rest);
                else
                    divmod_u64(last - large, (uint32_t)each, at, rest);
                parts = (uint32_t)at + (last < large ? 0 : more) - w + 1;
            }
            src.info[b * per_seq + hr] = make_uint2(slot, parts);
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const float s = over_groups(l[rt], [](float a, float b) { return a + b; });
            if (g == 0) {
                sh.ml[wave][rt * 16 + c][0] = m[rt];
                sh.ml[wave][rt * 16 + c][1] = s;
            }
        }
        __syncthreads();
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            float M = sh.ml[0][rt * 16 + c][0];
#pragma unroll
            for (int v = 1; v < kWaves; ++v) M = fmaxf(M, sh.ml[v][rt * 16 + c][0]);
            float a = exp2_fast(m[rt] - (M == kNegInf ? 0.0f : M));
            if (HALF) a *= __builtin_amdgcn_ldexpf(1.0f, E - kWeightExp);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int n = 0; n < NC; n += 4)
                    *reinterpret_cast<f32x4*>(&sh.os[rt][wave][c][channel_of<FMT, D>(g, r) + n]) =
                        f32x4{o[rt][n][r], o[rt][n + 1][r], o[rt][n + 2][r], o[rt][n + 3][r]} * a;
        }
        __syncthreads();
        const uint32_t row = threadIdx.x / 16, ch = threadIdx.x % 16 * NC;  // the thread's part of the outputs
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const uint32_t r = (rb * RT + rt) * 16 + row;
            float Mr = sh.ml[0][rt * 16 + row][0];
#pragma unroll
            for (int v = 1; v < kWaves; ++v) Mr = fmaxf(Mr, sh.ml[v][rt * 16 + row][0]);
            const float Mru = Mr == kNegInf ? 0.0f : Mr;
            float sum = 0.0f, y[NC];
#pragma unroll
            for (int n = 0; n < NC; ++n) y[n] = 0.0f;
#pragma unroll
            for (int v = 0; v < kWaves; ++v) {
                sum = fmaf(sh.ml[v][rt * 16 + row][1], exp2_fast(sh.ml[v][rt * 16 + row][0] - Mru), sum);
#pragma unroll
                for (int n = 0; n < NC; n += 4) {
                    const f32x4 z = *reinterpret_cast<const f32x4*>(&sh.os[rt][v][row][ch + n]);
                    y[n] += z.x;
                    y[n + 1] += z.y;
                    y[n + 2] += z.z;
                    y[n + 3] += z.w;
                }
            }
            if (FMT == kFmtPool) {
                fwht_row<NC>(y, lane);
                const float k = (float)((D == 128 ? 0.08838834764831845 : 0.125) / kLevelFactor);  // 1 / sqrt(d)
#pragma unroll
                for (int n = 0; n < NC; ++n) y[n] *= k;
            }
            if (r < src.rows) {
                if (whole && p.direct) {
                    uint32_t seq, qh;
                    row_of<FMT>(p, b, h, r, seq, qh);
                    // a row without tokens: zeros, and ln 0
                    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                    uint16_t* to = p.out.data + (uint64_t)seq * p.out.ts + (uint64_t)qh * p.out.hs + ch;
                    uint32_t z[NC / 2];
#pragma unroll
                    for (int n = 0; n < NC / 2; ++n) z[n] = pack_bf16x2(y[2 * n] * inv, y[2 * n + 1] * inv);
                    if constexpr (NC == 8)
                        *reinterpret_cast<uint4*>(to) = make_uint4(z[0], z[1], z[2], z[3]);
                    else
                        *reinterpret_cast<uint2*>(to) = make_uint2(z[0], z[1]);
                    if (p.lse && threadIdx.x % 16 == 0)
                        p.lse[(uint64_t)seq * p.Hq + qh] = (Mr + log2f(sum)) * 0.69314718055994531f;
                } else {
                    float* to = src.part + (uint64_t)slot * (16 * RT * (D + 2));
#pragma unroll
                    for (int n = 0; n < NC; n += 4)
                        *reinterpret_cast<f32x4*>(to + (rt * 16 + row) * D + ch + n) =
                            f32x4{y[n], y[n + 1], y[n + 2], y[n + 3]};
                    if (threadIdx.x % 16 == 0)
                        *reinterpret_cast<float2*>(to + 16 * RT * D + 2 * (rt * 16 + row)) = make_float2(Mr, sum);
                }
            }
        }
        if (left) __syncthreads();  // the next unit writes the same LDS
    }
}

template <int FMT, int D, int RT>
__global__ __launch_bounds__(kWaves* kWave, waves_per_simd(D, RT)) void attend_kernel(Common p, Source src) {
    fetch_arguments<sizeof(Common) + sizeof(Source)>();
    __shared__ Shared<D, RT> sh;
    attend_share<FMT, D, RT>(p, src, blockIdx.x, sh);
}

// A pool's workgroups and those of the tails behind it, in one launch.
template <int FMT, int D, int RT>
__global__ __launch_bounds__(kWaves* kWave, waves_per_simd(D, RT)) void attend_both_kernel(Common p, Source pool,
                                                                                           Source tail) {
    fetch_arguments<sizeof(Common) + 2 * sizeof(Source)>();
    __shared__ union {
        Shared<D, RT> a;
        Shared<D, 1> b;
    } sh;
    if (blockIdx.x < pool.W)
        attend_share<kFmtPool, D, RT>(p, pool, blockIdx.x, sh.a);
    else
        attend_share<FMT, D, 1>(p, tail, blockIdx.x - pool.W, sh.b);
}

// Joins the parts of a row: V waves a row, which take its parts in turn, d / 64
// channels a lane. What bounds it is latency, so a lane loads the maximum and
// sum of one part, and the parts' sums come eight at a time.
struct JoinParams {
    Common c;
    Source src[2];
    uint32_t rt[2];
    uint32_t sources;
};

template <int D, int V>
__global__ __launch_bounds__(kBlockThreads) void attend_join_kernel(JoinParams p) {
    fetch_arguments<sizeof(JoinParams)>();
    constexpr int C = D / 64, U = 8;
    constexpr int RPB = kBlockThreads / kWave / V;  // rows of a workgroup
    typedef float vec __attribute__((ext_vector_type(C)));
    const uint32_t lane = lane_id();
    const uint32_t wave = wave_uniform(threadIdx.x / kWave), w = wave % V;
    const uint32_t row = blockIdx.x * RPB + wave / V;
    if (row >= p.c.n * p.c.Hq) return;
    const uint32_t seq = row / p.c.Hq, qh = row % p.c.Hq;
    const uint32_t h = qh / p.c.group, i = qh % p.c.group;
    // this row's place in each source: its part k at from[s] + stride[s] * slot,
    // and the part's maximum and sum `ml` floats behind it
    const float* from[2] = {};
    uint32_t stride[2] = {}, ml[2] = {};
    u32x2 info[2] = {};  // first slot, number of parts
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        if ((uint32_t)s >= p.sources) break;
        const Source& x = p.src[s];
        const uint32_t tile = 16 * p.rt[s], r = x.pool ? seq * p.c.group + i : i, at = r % tile;
        // (a long pool's numbers could be worked out here: 0.6 us more than the load)
        info[s] = scalar_load<u32x2>(x.info + (x.pool ? 0 : seq * p.c.H * x.row_blocks) + h * x.row_blocks + r / tile);
        stride[s] = tile * (D + 2);
        from[s] = x.part + at * D;
        ml[s] = (tile - at) * D + at * 2;
    }
    const bool header = !p.src[0].pool || pool_header_ok(p.src[0], p.c.H, D);
    const uint32_t n0 = info[0].y, n = n0 + info[1].y;
    if (n == 0 || !header) return;  // written already, or never to be
    // this wave's parts w, w + V, ...: a lane has the place, maximum and sum of one of
    // each 64, and the first U parts' sums are on their way before the maxima are
    // needed (parts behind the last are read as the wave's first, or the row's)
    const uint32_t safe = w < n ? w : 0;
    const float* place;
    const auto ml_of = [&](uint32_t k) {
        k = k < n ? k : safe;
        const bool second = k >= n0;
        const uint32_t j = second ? k - n0 : k, slot = second ? info[1].x : info[0].x;
        place = (second ? from[1] : from[0]) + (uint64_t)(second ? stride[1] : stride[0]) * (j ? slot - 1 + 2 * j : slot);
        return *reinterpret_cast<const float2*>(place + (second ? ml[1] : ml[0]));
    };
    vec x[U];
    const auto load = [&](uint32_t j) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint64_t a = (uint64_t)place;
            const uint64_t lo = (uint32_t)__builtin_amdgcn_readlane((uint32_t)a, (j + u) & 63),
                           hi = (uint32_t)__builtin_amdgcn_readlane((uint32_t)(a >> 32), (j + u) & 63);
            x[u] = *((const __attribute__((address_space(1))) vec*)(lo | hi << 32) + lane);
        }
    };
    float2 v = ml_of(w + V * lane);
    load(0);
    float M = w + V * lane < n ? v.x : kNegInf, total = 0.0f;
    const bool many = n > w + V * kWave;  // more than one part a lane: `place` moves on
    for (uint32_t k = w + V * (lane + kWave); k < n; k += V * kWave) M = fmaxf(M, ml_of(k).x);
    M = last_lane(scan_wave(M, kNegInf, [](float a, float b) { return fmaxf(a, b); }));
    const float Mu = M == kNegInf ? 0.0f : M;
    vec y = 0.0f;
    for (uint32_t base = w; base < n; base += V * kWave) {
        const uint32_t k = base + V * lane;
        if (many) v = ml_of(k);
        const float a = exp2_fast(v.x - Mu);
        total = k < n ? fmaf(v.y, a, total) : total;
        const uint32_t rest = (n - base + V - 1) / V, count = rest < kWave ? rest : kWave;
        for (uint32_t j = 0; j < count; j += U) {
            if (j || many) load(j);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float f = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, a), (j + u) & 63));
                if (j + u < count) y += x[u] * f;
            }
        }
    }
    total = last_lane(scan_wave(total, 0.0f, [](float a, float b) { return a + b; }));
    if constexpr (V > 1) {
        __shared__ float mt[V][2];
        __shared__ vec ys[V][kWave];
        if (lane == 0) {
            mt[w][0] = M;
            mt[w][1] = total;
        }
        ys[w][lane] = y;
        __syncthreads();
        if (w) return;
        float all = M;
#pragma unroll
        for (int x = 1; x < V; ++x) all = fmaxf(all, mt[x][0]);
        const float allu = all == kNegInf ? 0.0f : all;
        total = 0.0f;
        y = 0.0f;
#pragma unroll
        for (int x = 0; x < V; ++x) {
            const float a = exp2_fast(mt[x][0] - allu);
            total = fmaf(mt[x][1], a, total);
            y += ys[x][lane] * a;
        }
        M = all;
    }
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    uint16_t* to = p.c.out.data + (uint64_t)seq * p.c.out.ts + (uint64_t)qh * p.c.out.hs;
    if constexpr (C == 2)
        reinterpret_cast<uint32_t*>(to)[lane] = pack_bf16x2(y.x * inv, y.y * inv);
    else
        to[lane] = (uint16_t)pack_bf16x2(y.x * inv, 0.0f);
    if (p.c.lse && lane == 0) p.c.lse[row] = (M + log2f(total)) * 0.69314718055994531f;
}

// A workgroup gets at least kMinBlocks blocks of sequences as long as their table is wide: half a launch's latency
// goes into starting a share and joining it (a 4096-token pool for 15 agents, alone and with tails: 17.3 and 20.8
// us with 1, 13.7 and 15.2 with 2, 14.7 and 15.4 with 4). The host knows no lengths: far shorter sequences are
// shared out a block each (one of 100 tokens 5.0 us, with a table eight times as wide as it needs 7.3).
// Up to kWholeTokens tokens a unit stays whole and its outputs need no second launch: 1, 15 and 64 sequences of 512
// tokens (8 kv heads of 128, int8) 8.5, 8.8 and 14.9 us, cut up 9.7, 10.2 and 17.5; of 1024 12.3, 13.7 and 24.2,
// cut up 9.8, 12.7 and 26.9.
constexpr uint64_t kMinBlocks = 2, kWholeTokens = 512;

// The plan with rt row tiles a wave.
AttendPlan plan_of(uint64_t units_of_rows, uint32_t rows, uint64_t max_tokens, uint32_t d, uint32_t rt, bool direct) {
    AttendPlan a;
    a.rows = rows;
    a.rt = rt;
    a.row_blocks = (rows + 16 * rt - 1) / (16 * rt);
    a.units = units_of_rows * a.row_blocks;
    const uint64_t slots = 256ull * waves_per_simd(d, rt);
    a.blocks = a.units * ((max_tokens + kBlock - 1) / kBlock);
    // Eight units for each place of a workgroup balance one another, whatever their lengths, but for a single
    // long one: 512 sequences (8 kv heads of 128, int8) of 1024 tokens 182 us, cut up 202; of 1 to 2048 197 and
    // 245; one of 32768 among 511 of 100 tokens 250 and 62.
    a.whole = max_tokens <= kWholeTokens || a.units >= 8 * slots;
    uint64_t w = a.blocks / kMinBlocks < slots ? a.blocks / kMinBlocks : slots;
    if (w < 1) w = 1;
    a.W = a.whole ? a.units : w;
    a.slots = a.whole ? (direct ? 0 : a.units) : 2 * w + (direct ? 0 : a.units);
    // what the workspace has room for: that of a plan that is cut up, unless no sequence is long enough for one,
    // and of one row tile a wave, which fewer rows or tokens would take
    const uint64_t room = max_tokens <= kWholeTokens ? a.slots : 2 * w + (direct ? 0 : a.units);
    a.room = a.bytes_of(room, d);
    if (rt > 1) {
        const uint64_t one = plan_of(units_of_rows, rows, max_tokens, d, 1, direct).room;
        if (one > a.room) a.room = one;
    }
    return a;
}

// one_tile: up to so many rows are taken one row tile a wave.
AttendPlan make_plan(uint64_t units_of_rows, uint32_t rows, uint64_t max_tokens, uint32_t d, uint32_t one_tile,
                     bool direct) {
    // Two row tiles of a wave share the widening of the tokens, but start and
    // join later: taken where every workgroup has a block to do. A call with two and
    // with one, over the same inputs again and again (which the 256 MB cache then holds; a
    // pool of 131071 tokens that it does not hold takes 78), us: pool of 15 agents, 60 rows, heads of 128:
    // 131071 tokens 70 and 103, 4096 with tails 15.2 and 18.0, 1024 11.5 and 9.7. Pages, 8
    // sequences of 8192, 2 kv heads: heads of 64, 17 rows int8 12.4 and 13.0, bf16 12.0 and
    // 15.6; heads of 128, int8 32 rows 19.9 and 17.0, 48 rows 21.6 and 25.3, bf16 27.3
    // and 37.3 (where 44 vector registers are spilled).
    const uint64_t most_blocks = (max_tokens + kBlock - 1) / kBlock;
    const bool enough = units_of_rows * ((rows + 31) / 32) * most_blocks >= 256ull * waves_per_simd(d, 2);
    return plan_of(units_of_rows, rows, max_tokens, d, rows > one_tile && enough ? 2 : 1, direct);
}

template <int D>
hipError_t launch_pages(uint32_t format, uint32_t rt, uint32_t grid, const Common& p, const Source& s, hipStream_t stream) {
    const auto f = format == 0   ? (rt == 1 ? attend_kernel<kFmtBf16, D, 1> : attend_kernel<kFmtBf16, D, 2>)
                   : format == 1 ? (rt == 1 ? attend_kernel<kFmtInt8, D, 1> : attend_kernel<kFmtInt8, D, 2>)
                                 : (rt == 1 ? attend_kernel<kFmtFp8, D, 1> : attend_kernel<kFmtFp8, D, 2>);
    return launch_kernel(f, dim3(grid), dim3(kWaves * kWave), stream, p, s);
}
template <int D>
hipError_t launch_both(uint32_t format, uint32_t rt, uint32_t grid, const Common& p, const Source& a, const Source& b,
                       hipStream_t stream) {
    const auto f = format == 0   ? (rt == 1 ? attend_both_kernel<kFmtBf16, D, 1> : attend_both_kernel<kFmtBf16, D, 2>)
                   : format == 1 ? (rt == 1 ? attend_both_kernel<kFmtInt8, D, 1> : attend_both_kernel<kFmtInt8, D, 2>)
                                 : (rt == 1 ? attend_both_kernel<kFmtFp8, D, 1> : attend_both_kernel<kFmtFp8, D, 2>);
    return launch_kernel(f, dim3(grid), dim3(kWaves * kWave), stream, p, a, b);
}

// The source's share of the workspace, and the bytes it takes.
uint64_t place_source(Source& s, const AttendPlan& plan, uint32_t d, uint8_t* ws) {
    s.rows = plan.rows;
    s.row_blocks = plan.row_blocks;
    s.W = (uint32_t)plan.W;
    s.whole = plan.whole;
    s.part = reinterpret_cast<float*>(ws);
    s.info = reinterpret_cast<uint2*>(ws + plan.part_bytes(d));
    return plan.bytes(d);
}

}  // namespace

AttendPlan page_attend_plan(uint32_t n_seqs, uint32_t H, uint32_t Hq, uint32_t d, uint64_t max_tokens, bool tail) {
    return make_plan((uint64_t)n_seqs * H, Hq / H, max_tokens, d, tail ? ~0u : d == 64 ? 16 : 32, !tail);
}

AttendPlan pool_attend_plan(uint32_t H, uint32_t n_agents, uint32_t Hq, uint32_t d, uint32_t T, bool tail) {
    return make_plan(H, n_agents * (Hq / H), T, d, 16, !tail);
}

hipError_t launch_attend(const AttendArgs& a, hipStream_t stream) {
    Common p{};
    p.q = a.q;
    p.out = a.out;
    p.lse = a.lse;
    p.status = a.status;
    p.n = a.n;
    p.H = a.H;
    p.Hq = a.Hq;
    p.group = a.Hq / a.H;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    const bool has_pool = a.pool != nullptr, has_pages = a.tail.table != nullptr;
    p.direct = !(has_pool && has_pages);
    uint8_t* ws = static_cast<uint8_t*>(a.ws);
    AttendPlan pool_plan{}, page_plan{};
    Source pool{}, pages{};
    if (has_pool) {
        pool_plan = pool_attend_plan(a.H, a.n, a.Hq, a.d, a.T, has_pages);
        ws += place_source(pool, pool_plan, a.d, ws);
        pool.pool = a.pool;
        pool.lay = pool_layout(a.L, a.H, a.T, a.d);
        pool.L = a.L;
        pool.T = a.T;
        pool.layer = a.layer;
        const uint64_t total = pool_plan.units * ((a.T + kBlock - 1) / kBlock);
        pool.each = total / pool_plan.W;
        pool.more = (uint32_t)(total % pool_plan.W);
    }
    if (has_pages) {
        const PageLayout& lay = a.tail.lay;
        page_plan = page_attend_plan(a.n, a.H, a.Hq, a.d, (uint64_t)a.tail.table_cols * lay.P, has_pool);
        ws += place_source(pages, page_plan, a.d, ws);
        pages.pages = a.tail.pages;
        pages.table = a.tail.table;
        pages.table_stride = a.tail.table_stride;
        pages.lens = a.tail.lens;
        pages.table_cols = a.tail.table_cols;
        pages.num_pages = lay.num_pages;
        pages.page_shift = 31 - __builtin_clz(lay.P);
        pages.page_bytes = lay.page_bytes;
        pages.steps = lay.steps;
    }
    hipError_t e;
    if (has_pool && has_pages) {
        const uint32_t grid = pool.W + pages.W;
        e = a.d == 64 ? launch_both<64>(a.tail.lay.format, pool_plan.rt, grid, p, pool, pages, stream)
                      : launch_both<128>(a.tail.lay.format, pool_plan.rt, grid, p, pool, pages, stream);
    } else if (has_pool) {
        const auto f = a.d == 64 ? (pool_plan.rt == 1 ? attend_kernel<kFmtPool, 64, 1> : attend_kernel<kFmtPool, 64, 2>)
                                 : (pool_plan.rt == 1 ? attend_kernel<kFmtPool, 128, 1> : attend_kernel<kFmtPool, 128, 2>);
        e = launch_kernel(f, dim3(pool.W), dim3(kWaves * kWave), stream, p, pool);
    } else {
        e = a.d == 64 ? launch_pages<64>(a.tail.lay.format, page_plan.rt, pages.W, p, pages, stream)
                      : launch_pages<128>(a.tail.lay.format, page_plan.rt, pages.W, p, pages, stream);
    }
    const AttendPlan& first = has_pool ? pool_plan : page_plan;
    if (e != hipSuccess || (p.direct && first.whole)) return e;
    JoinParams j{};
    j.c = p;
    j.src[0] = has_pool ? pool : pages;
    j.rt[0] = first.rt;
    j.src[1] = pages;
    j.rt[1] = has_pages ? page_plan.rt : 1;
    j.sources = p.direct ? 1 : 2;
    const uint64_t rows = (uint64_t)a.n * a.Hq;
    // One wave joins a row of few parts, four one of many. A call with one and with four, us: pages of 1, 4, 8, 15
    // and 32 sequences of 4096 tokens (W / units 64, 16, 8, 4, 2) 10.4 and 10.0, 13.4 and 13.1, 18.3 and 18.6, 28.8
    // and 29.2, 48.0 and 48.7; a pool of 8192 tokens for 4 agents (32) 12.2 and 10.7, of 131071 over 2 kv heads (256) 32.9
    // and 19.9. It goes by the mean: of 100 sequences (5) one of 40000 tokens among 99 of 100 takes 31.2, with four 16.4.
    const bool few = first.whole || first.W <= 6 * first.units;
    if (few)
        return launch_kernel(a.d == 64 ? attend_join_kernel<64, 1> : attend_join_kernel<128, 1>,
                             dim3((uint32_t)((rows + 3) / 4)), dim3(kBlockThreads), stream, j);
    return launch_kernel(a.d == 64 ? attend_join_kernel<64, 4> : attend_join_kernel<128, 4>, dim3((uint32_t)rows),
                         dim3(kBlockThreads), stream, j);
}

}  // namespace kvc
