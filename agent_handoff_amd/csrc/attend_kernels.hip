// attend_kernels.hip - attention of one new token (over pages also with a window, or
// of a few) over a paged cache or one layer of the shared pool, for gfx950.
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
// 4-bit pages: a code times its power of two is a bf16 number, so both products are
// bf16's, and the byte that follows the codes is all that a vector needs. 32 sequences as above: 57 us, 5.0 TB/s; half
// the bytes of 8 bits, but as many instructions for as many tokens (a SIMD's VALU is busy half of the time).
// A window: a sequence's tokens are counted without the gap between its sinks and its
// window, cut out in whole runs of 16, so nothing between is read (int8, 32 sequences of up to 16384 tokens, window
// 4096: 49 us, 4.9 TB/s; one of 5000 tokens, window 1024: 10 us of latency and 4 of joining, where the length has to
// be known before the table is read).
// Few new tokens of each sequence: its rows are tokens times heads, each with a position of its
// own, which masks single tiles at the ends; what bounds it is still memory (15 sequences of 5 drafts behind 8192
// tokens, e4m3, 20 rows: 60 us, 4.3 TB/s).
//
// Tried and left out: keeping two tiles of loads in registers (spills, or the same
// time; in LDS, see through_lds); sharing widened tokens among the waves through LDS (a quarter fewer
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
#include "lds_fetch.h"
#include "page_codes.h"

#include <type_traits>

namespace kvc {
namespace {

constexpr int kDevBadHeader = 1, kDevBadPage = 32, kDevBadLength = 64, kDevBadStart = 128;  // KVC_DEV_*
constexpr int kFmtBf16 = kPageBf16, kFmtInt8 = kPageInt8, kFmtFp8 = kPageFp8, kFmtFp4 = kPageFp4, kFmtPool = 3;
// Products in binary16 (codes of 8 bits, levels) or in bf16 (which holds a 4-bit code times its power of two exactly).
constexpr bool half_products(int fmt) { return fmt != kFmtBf16 && fmt != kFmtFp4; }
constexpr int kWaves = 4;
constexpr uint32_t kTile = 32;
constexpr uint32_t kBlock = kWaves * kTile;  // tokens of one step of a workgroup
constexpr uint32_t kPageRun = 32 * kBlock;   // 32 tiles a wave: a page number for 16 tokens in each of 64 lanes
constexpr float kSlack = 3.0f;
constexpr int kWeightExp = 12;
constexpr int kMinExp = -100;  // steps below 2^-100 are taken with this exponent
constexpr float kNegInf = -__builtin_inff();
// What a kernel is compiled for: one new token of each sequence that sees all of it; or a window and sinks; or many new
// tokens, each of which sees those up to its own (with a window or without).
constexpr int kOneSeesAll = 0, kOneWindow = 1, kMany = 2;

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
    union {
        uint32_t L;
        uint32_t window;  // pages with a window
    };
    union {
        uint32_t T;
        uint32_t sinks;
    };
    uint32_t layer;
    union {
        uint32_t more;    // shares of `each` blocks, the first `more` of them one larger
        uint32_t tokens;  // many new tokens: query rows, of
    };
    union {
        uint64_t each;
        const int32_t* starts;  // sequence b: starts[b] to starts[b + 1] - 1
    };
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
// The top bit of each half that holds a bf16 that is not finite.
__device__ __forceinline__ uint32_t infinite(uint32_t v) { return ((v & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }
template <int FMT>
__device__ __forceinline__ f32x4 mfma(const u32x4& a, const u32x4& b, const f32x4& c) {
    return half_products(FMT) ? mfma_half(a, b, c) : mfma_bf16(a, b, c);
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

template <int D>
struct Raw<kFmtFp4, D> {
    uint32_t k[2][D / 32];   // the lane's quarter of a key's codes
    uint32_t kp[2];          // its power of two
    uint32_t v[8];           // D / 16 codes of a value
    uint32_t vp[2][D / 32];  // powers of the four tokens of a run, D / 32 bytes each
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

__device__ __forceinline__ void take_steps(const uint8_t* from, float* to) {
    const float4 a = *reinterpret_cast<const float4*>(from);
    to[0] = a.x;
    to[1] = a.y;
    to[2] = a.z;
    to[3] = a.w;
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
// What a new token sees of `len` tokens with a window and sinks: tokens below
// min(sinks, lo) and from lo = len - window on. The gap between them is cut out
// in whole runs of 16, so that runs stay inside pages: tokens are counted without it
// (`len` of them), and those from hid0 to hid1, less than two runs, do not count.
struct Seen {
    uint32_t len, hid0, hid1;
    uint32_t cut, gap;  // token t stands for t + gap from `cut` on
};
// (of many new tokens: what any of them sees)
template <int MODE>
__device__ __forceinline__ Seen seen_of(const Source& p, uint32_t len, uint32_t tokens = 1) {
    Seen s{len, 0, 0, 0, 0};
    if (MODE == kOneSeesAll || (MODE == kMany && p.window == 0)) return s;
    const uint32_t back = p.window + tokens - 1, lo = len > back ? len - back : 0;
    s.hid0 = p.sinks < lo ? p.sinks : lo;
    s.cut = (s.hid0 + 15) & ~15u;
    s.gap = (lo & ~15u) > s.cut ? (lo & ~15u) - s.cut : 0;
    s.len = len - s.gap;
    s.hid1 = lo - s.gap;
    return s;
}
// Blocks of a length; an empty sequence has one, without tokens.
__device__ __forceinline__ uint32_t blocks_of(uint32_t len) { return len <= kBlock ? 1 : (len + kBlock - 1) / kBlock; }

// The new tokens of sequence b (many new tokens), none where its starts are wrong.
struct Fresh {
    uint32_t first, count;
    bool bad;
};
__device__ __forceinline__ Fresh fresh_of(const Source& p, uint32_t b) {
    const int32_t a = p.starts[b], e = p.starts[b + 1];
    const bool bad = a < 0 || e < a || (uint32_t)e > p.tokens;
    return Fresh{bad ? 0u : (uint32_t)a, bad ? 0u : (uint32_t)(e - a), bad};
}
// Row blocks of a kv head for so many new tokens; and the place of a sequence's first in the list of units (those of
// the sequences before it, rounded up one by one, are no more).
template <int RT>
__device__ __forceinline__ uint32_t row_blocks_of(uint32_t count, uint32_t group) {
    return (count * group + 16 * RT - 1) / (16 * RT);
}
template <int RT>
__device__ __forceinline__ uint64_t first_unit(uint32_t b, uint32_t first, uint32_t group, uint32_t H) {
    return (uint64_t)(first * group / (16 * RT) + b) * H;
}

// Which tokens a query row sees, counted from where its lane's tokens of a run begin.
struct Sight {
    int32_t past, left, sunk_to;
    __device__ __forceinline__ bool operator()(int32_t c) const { return (c <= past) & ((c > left) | (c < sunk_to)); }
};

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

// Tiles on their way to a wave lie in its registers, or in LDS, which a wave fills for itself. In LDS they cost more
// instructions, but leave registers for a second row tile of heads of 128, where bf16's spill otherwise, and 8 bits' too
// if there is a window or each row has a position of its own. (8 kv heads of 128, us in registers and in LDS. One new token,
// 40 rows: bf16, 15 sequences of 400 tokens 14.5 and 12.8, 4 of 2000 21.8 and 17.1, 64 of 1000 103 and 92, 32 of 8000 300
// and 310; e4m3 10.7 and 11.3, 18.1 and 18.5, 52.4 and 53.5, 155 and 164. Windows: bf16, 4 sequences of 1024 tokens 27.5
// and 20.0, 32 of 4096 164 and 159; e4m3 22.0 and 20.1, 64 of 1000 56.6 and 54.1, 32 of 4096 89.8 and 92.0. 15 sequences of 5
// drafts behind 8192 tokens: bf16 135 and 104, e4m3 73.0 and 66.0. Heads of 64, whose registers suffice, e4m3: 64 sequences of
// 1000 tokens, 20 rows, 19.7 and 23.7; those drafts 39.2 and 42.9. 4 bits, those drafts with heads of 128: 54 and 58.) One row
// tile needs no room: 32 windows of 4096 int8 52 and 55, bf16 98 and 97, 32 sequences of up to 16384 in 4 bits 61 and 69.
constexpr bool through_lds(int fmt, int d, int rt, int mode) {
    const bool bits8 = fmt == kFmtInt8 || fmt == kFmtFp8;
    return rt == 2 && d == 128 && (fmt == kFmtBf16 || (bits8 && mode != kOneSeesAll));
}

// A tile: rows of keys, of values, then the steps of both. The keys' chunks of 16 bytes change places inside a row by
// the token, so that 16 lanes with one chunk of 16 tokens meet in no bank.
template <int FMT, int D, int RT>
struct Ring {
    static constexpr uint32_t kRow = page_code_bytes(FMT, D), kCodes = kTile * kRow;
    static constexpr uint32_t kBytes = 2 * kCodes + 2 * kTile * page_step_bytes(FMT, D);
    static constexpr uint32_t kRunLoads = kRow / 64;  // of 16 tokens
    static constexpr uint32_t kLoads = 4 * kRunLoads + (page_step_bytes(FMT, D) ? 1 : 0);
    static constexpr uint32_t kRoom = 160 * 1024 / waves_per_simd(D, RT) - 2048;  // the rest of Shared is smaller
    static constexpr uint32_t kDepth = kRoom / (kWaves * kBytes);
    static_assert(kDepth >= 1 && kLoads * (kDepth - 1) < 64);
    static __device__ __forceinline__ uint32_t turn(uint32_t token) {
        return kRow == 256 ? token & 15 : kRow == 128 ? token >> 1 & 7 : token >> 2 & 3;
    }
    uint8_t tile[kWaves][kDepth][kBytes];
};
struct NoRing {};

// LDS of a workgroup. (Without its alignment, accesses of four floats come out in pairs.)
template <int FMT, int D, int RT, int MODE>
struct Shared {
    alignas(16) float ml[kWaves][RT * 16][2];
    union {
        alignas(16) float os[RT][kWaves][16][D + 4];
        alignas(16) std::conditional_t<through_lds(FMT, D, RT, MODE), Ring<FMT, D, RT>, NoRing> ring;
    };
    uint32_t sums[kWaves];
    uint32_t found[3];  // sequence, blocks before it, its blocks
};

// Tiles that are on their way at once.
template <int FMT, int D, int RT, int MODE>
constexpr uint32_t ahead_of() {
    if constexpr (through_lds(FMT, D, RT, MODE))
        return Ring<FMT, D, RT>::kDepth;
    else
        return 1;
}

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
template <int FMT, int D, int RT, int MODE>
__device__ __forceinline__ void attend_share(const Common& p, const Source& src, uint32_t w, Shared<FMT, D, RT, MODE>& sh) {
    constexpr int KS = D / 32;   // key product steps
    constexpr int NC = D / 16;   // channels of a lane, value products
    constexpr bool HALF = half_products(FMT);
    constexpr bool MANY = MODE == kMany, WIN = MODE != kOneSeesAll;
    constexpr bool RING = through_lds(FMT, D, RT, MODE);
    constexpr int RE = MANY ? RT : 1;  // exponents taken out of the weights: of a row, where rows see different tokens
    using R = Raw<FMT, D>;
    const uint32_t lane = lane_id(), c = lane & 15, g = lane >> 4;
    const uint32_t wave = wave_uniform(threadIdx.x / kWave);
    const uint32_t per_seq = MANY ? p.H : p.H * src.row_blocks;  // units of a sequence (that share a row block)
    // what a sequence adds to the list of blocks, over `per_seq`
    const auto weight_of = [&](uint32_t s) {
        const int32_t given = src.lens[s];
        const uint32_t len = clamp_length(src, given);
        if (!MANY) return blocks_of(seen_of<MODE>(src, len).len);
        const Fresh x = fresh_of(src, s);
        if (w == 0 && p.status && (x.bad || bad_length(src, given)))
            atomicOr(p.status, (x.bad ? kDevBadStart : 0) | (bad_length(src, given) ? kDevBadLength : 0));
        return row_blocks_of<RT>(x.count, p.group) * blocks_of(seen_of<MODE>(src, len, x.count).len);
    };

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
            const uint32_t v = lane < p.n ? weight_of(lane) : 0;
            // (wrong starts could give rows many times over: nothing is done)
            if (MANY && __ballot(lane < p.n && fresh_of(src, lane).bad) != 0) return;
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
            bool bad = false;
            for (uint32_t s = s0; s < s1; ++s) {
                v += weight_of(s);
                if (MANY) bad |= fresh_of(src, s).bad;
            }
            if (MANY && __syncthreads_or(bad)) return;
            const uint32_t at0 = scan_threads(v, sh.sums, all);
            if (!share((uint64_t)wave_uniform(all) * per_seq)) return;
            divmod_u64(x0, per_seq, q64, part);
            const uint32_t q = (uint32_t)q64;
            if (q >= at0 && q - at0 < v) {
                uint32_t at = at0, s = s0, nb = 0;
                for (; s < s1; ++s) {
                    nb = weight_of(s);
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
        if (MANY) {
            const uint32_t count = fresh_of(src, b).count;
            mine /= row_blocks_of<RT>(count, p.group);
        }
        divmod_u64(x0 - (uint64_t)before * per_seq, mine, q64, off);
        hr = (uint32_t)q64;
    }

    uint64_t first = x0 - off;  // the unit's first block
    for (uint32_t nb = 0; left != 0; off = 0, ++hr, first += nb) {
        Fresh fresh{};
        uint32_t row_blocks = src.row_blocks, rows = src.rows;
        if constexpr (MANY) {
            for (;; hr = 0, ++b) {
                if (b >= p.n) return;
                fresh = fresh_of(src, b);
                fresh.first = wave_uniform(fresh.first);
                fresh.count = wave_uniform(fresh.count);
                row_blocks = row_blocks_of<RT>(fresh.count, p.group);
                rows = fresh.count * p.group;
                if (hr < p.H * row_blocks) break;
            }
        } else {
            if (FMT != kFmtPool && hr == per_seq) {
                hr = 0;
                ++b;
            }
            if (FMT == kFmtPool ? hr >= per_seq : b >= p.n) break;
        }
        const uint64_t unit = MANY ? first_unit<RT>(b, fresh.first, p.group, p.H) + hr : b * per_seq + hr;
        const uint32_t h = hr / row_blocks, rb = hr % row_blocks;
        // query row r of the unit's
        const auto place_of = [&](uint32_t r, uint32_t& at, uint32_t& qh) {
            if (MANY) {
                at = fresh.first + r / p.group;
                qh = h * p.group + r % p.group;
            } else {
                row_of<FMT>(p, b, h, r, at, qh);
            }
        };

        // everything that can be asked for at once: the queries (row 16 rt + c,
        // channels as the key loads have them), the length, the first page numbers
        uint32_t qw[RT][KS][4];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const uint32_t r = (rb * RT + rt) * 16 + c;
            uint32_t seq, qh;
            place_of(r < rows ? r : 0, seq, qh);
            const uint8_t* qp = reinterpret_cast<const uint8_t*>(p.q.data + (uint64_t)seq * p.q.ts + (uint64_t)qh * p.q.hs);
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const uint32_t ch = FMT == kFmtFp4 ? g * (D / 4) + s * 8
                                    : HALF         ? (s / 2) * 64 + g * 16 + (s % 2) * 8
                                                   : s * 32 + g * 8;
                load_words(qp + 2 * ch, qw[rt][s]);
            }
        }
        // page numbers of this wave's 16-token runs: run i of tile t in lane 2t + i
        // (whole rows of the table can be read, whatever the length)
        const uint32_t run0 = ((lane >> 1) * kWaves + wave) * kTile + (lane & 1) * 16;
        Seen seen{};
        const auto real = [&](uint32_t t) { return WIN && t >= seen.cut ? t + seen.gap : t; };
        const auto load_pages = [&](uint32_t base) {
            const uint32_t t = real(base + run0) >> src.page_shift;
            return src.table[b * src.table_stride + (t < src.table_cols ? t : 0)];
        };
        int32_t given = 0, page = 0;
        if (FMT != kFmtPool) {
            given = src.lens[b];
            if (!WIN) page = load_pages(off * kBlock);
        }
        const uint32_t length = FMT == kFmtPool ? src.T : wave_uniform(clamp_length(src, given));
        seen = seen_of<MODE>(src, length, MANY ? fresh.count : 1);
        // many new tokens: each row's position, and the tokens that all of them see
        int32_t pos[MANY ? RT : 1];
        uint32_t all_from = seen.hid1, all_to = seen.len;
        if constexpr (MANY) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const uint32_t r = (rb * RT + rt) * 16 + c;
                pos[rt] = (int32_t)length - (int32_t)fresh.count + (int32_t)((r < rows ? r : 0) / p.group);
            }
            const uint32_t last = src.window && length > src.window ? length - src.window : 0;
            all_from = last > seen.gap ? last - seen.gap : 0;
            all_to = length + 1 > fresh.count + seen.gap ? length + 1 - fresh.count - seen.gap : 0;
        }
        if (WIN) page = load_pages(off * kBlock);
        const uint32_t len = seen.len;
        if (FMT != kFmtPool && !MANY && hr == 0 && off == 0 && threadIdx.x == 0 && bad_length(src, given) && p.status)
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
            } else if constexpr (!RING) {
                constexpr uint32_t ROW = page_code_bytes(FMT, D);
                const uint32_t P = 1u << src.page_shift;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t pg = __builtin_amdgcn_readlane(my_page, (2 * it + i) & 63);
                    const uint8_t* pb = src.pages + (uint64_t)pg * src.page_bytes;
                    const uint32_t at = real(t0 + 16 * i) & (P - 1);
                    const uint32_t kl = h * P + at, vl = (p.H + h) * P + at;  // rows inside the page
                    const uint8_t* kb = pb + (uint64_t)kl * ROW;
                    const uint8_t* vb = pb + (uint64_t)vl * ROW;
                    if constexpr (FMT == kFmtFp4) {
                        constexpr uint32_t PB = D / kFp4Block;  // powers of a vector
                        const uint8_t* sb = pb + src.steps;
                        load_words(kb + c * ROW + g * (ROW / 4), x.k[i]);
                        x.kp[i] = sb[(uint64_t)(kl + c) * PB + g / (4 / PB)];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint8_t* va = vb + (4 * g + j) * ROW + c * (ROW / 16);
                            x.v[4 * i + j] = D == 128 ? *reinterpret_cast<const uint32_t*>(va) : *reinterpret_cast<const uint16_t*>(va);
                        }
                        load_words(sb + (uint64_t)(vl + 4 * g) * PB, x.vp[i]);
                    } else {
#pragma unroll
                        for (int s = 0; s < R::KL; ++s)
                            x.k[i][s] = *reinterpret_cast<const uint4*>(kb + c * ROW + 64 * s + 16 * g);
#pragma unroll
                        for (int j = 0; j < 4; ++j) load_words(vb + (4 * g + j) * ROW + c * (ROW / 16), x.v[4 * i + j]);
                        if (FMT != kFmtBf16) {
                            take_steps(pb + src.steps + (uint64_t)(kl + 4 * g) * 4, &x.ks[4 * i]);
                            take_steps(pb + src.steps + (uint64_t)(vl + 4 * g) * 4, &x.vs[4 * i]);
                        }
                    }
                }
            } else {
                using Way = Ring<FMT, D, RT>;
                constexpr uint32_t ROW = Way::kRow, STEP = page_step_bytes(FMT, D), N = Way::kRunLoads;
                const uint32_t P = 1u << src.page_shift;
                uint8_t* to = sh.ring.tile[wave][it % Way::kDepth];
                const uint8_t *k[2], *v[2], *steps[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t pg = __builtin_amdgcn_readlane(my_page, (2 * it + i) & 63);
                    const uint8_t* pb = src.pages + (uint64_t)pg * src.page_bytes;
                    const uint32_t kl = h * P + (real(t0 + 16 * i) & (P - 1));  // row inside the page
                    k[i] = pb + (uint64_t)kl * ROW;
                    v[i] = pb + (uint64_t)(kl + p.H * P) * ROW;
                    steps[i] = pb + src.steps + (uint64_t)kl * STEP;
                }
                // (what was read of the buffer has arrived)
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                uint32_t ko[N], vo[N];
#pragma unroll
                for (uint32_t u = 0; u < N; ++u) {
                    constexpr uint32_t CPR = ROW / 16;  // chunks of a row
                    ko[u] = lane / CPR * ROW + (lane % CPR ^ Way::turn(u * (64 / CPR) + lane / CPR)) * 16;
                    vo[u] = lane * 16;
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) fetch16<N>(k[i], ko, to + 16 * i * ROW);
#pragma unroll
                for (int i = 0; i < 2; ++i) fetch16<N>(v[i], vo, to + Way::kCodes + 16 * i * ROW);
                // keys' steps of both runs, then values'
                if constexpr (STEP != 0)
                    fetch_lane4((lane & 16 ? steps[1] : steps[0]) + (lane & 32 ? (uint64_t)p.H * P * STEP : 0) + lane % 16 * 4,
                                to + 2 * Way::kCodes);
            }
        };
        // a tile's keys, and its values and steps, out of LDS; it is waited for while `behind` tiles may be on their way
        const auto take_keys = [&](uint32_t it, uint32_t behind, R& x) {
            if constexpr (RING) {
                using Way = Ring<FMT, D, RT>;
                wait_loads<Way::kLoads, Way::kDepth - 1>(behind);
                const uint8_t* at = sh.ring.tile[wave][it % Way::kDepth];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (uint32_t s = 0; s < (uint32_t)R::KL; ++s)
                        x.k[i][s] = *reinterpret_cast<const uint4*>(at + (16 * i + c) * Way::kRow + ((4 * s + g) ^ Way::turn(c)) * 16);
            }
        };
        const auto take_values = [&](uint32_t it, R& x) {
            if constexpr (RING) {
                using Way = Ring<FMT, D, RT>;
                const uint8_t* at = sh.ring.tile[wave][it % Way::kDepth] + Way::kCodes;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        load_words(at + (16 * i + 4 * g + j) * Way::kRow + c * (Way::kRow / 16), x.v[4 * i + j]);
                    if constexpr (FMT != kFmtBf16) {
                        const uint8_t* steps = at + Way::kCodes;
                        take_steps(steps + (16 * i + 4 * g) * 4, &x.ks[4 * i]);
                        take_steps(steps + (kTile + 16 * i + 4 * g) * 4, &x.vs[4 * i]);
                    }
                }
            }
        };
        R x;
        // the first tiles from `base` on: as many as there is room for
        constexpr uint32_t kAhead = ahead_of<FMT, D, RT, MODE>();
        const auto load_first = [&](uint32_t base) {
            const uint32_t stop = FMT == kFmtPool || end - base <= kPageRun ? end : base + kPageRun;
#pragma unroll
            for (uint32_t u = 0; u < kAhead; ++u)
                if (base + wave * kTile + u * kBlock < stop) load(base + wave * kTile + u * kBlock, u, x);
        };
        load_first(begin);
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
            const bool live = (rb * RT + rt) * 16 + c < rows;
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
        int E[RE];  // exponent taken out of the weights (HALF)
        float elimit[RE], wmul[RE];  // 2^E, which no step so far has reached; 2^(kWeightExp - E)
#pragma unroll
        for (int e = 0; e < RE; ++e) {
            E[e] = kMinExp;
            elimit[e] = __builtin_amdgcn_ldexpf(1.0f, kMinExp);
            wmul[e] = __builtin_amdgcn_ldexpf(1.0f, kWeightExp - kMinExp);
        }
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

        // whether the lane's token j of a tile at t0 counts
        const auto counts = [&](uint32_t t0, int j) {
            const uint32_t t = t0 + (j < 4 ? 0 : 16) + 4 * g + (j & 3);
            return WIN ? t < end && (t < seen.hid0 || t >= seen.hid1) : t < end;
        };
        // One tile: its loads are in x, or on their way to LDS; those of a later one (if it lies before `stop`) go
        // out as soon as x has been widened, or read. PART: some of its tokens do not count.
        const auto tile = [&](auto part, uint32_t t0, uint32_t stop, uint32_t it, R& x) {
            constexpr bool PART = decltype(part)::value;
            constexpr bool LAST = PART && !WIN;  // none lies behind it
            take_keys(it, (stop - t0 - 1) / kBlock, x);
            f32x4 s[RT][2];
            {
                u32x4 kf[2][KS];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        if constexpr (FMT == kFmtFp4) {
                            const uint32_t y = x.k[i][k], p2 = x.kp[i] << 23;
                            kf[i][k] = u32x4{widen_fp4<0>(y, p2), widen_fp4<1>(y, p2), widen_fp4<2>(y, p2), widen_fp4<3>(y, p2)};
                        } else if constexpr (HALF) {
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
            take_values(it, x);
            if (RING && !LAST && t0 + kAhead * kBlock < stop) load(t0 + kAhead * kBlock, it + kAhead, x);
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
            } else if constexpr (FMT == kFmtFp4) {
                constexpr int PB = D / kFp4Block;
                if (PART) {  // as below; a power that no token wrote may be NaN, times a code of 0 too
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const bool ok = counts(t0, j);
                        x.v[j] = ok ? x.v[j] : 0;
                        uint32_t& w = x.vp[j >> 2][(j & 3) * PB / 4];
                        const uint32_t none = w & ~((PB == 4 ? ~0u : 0xFFFFu) << ((j & 3) * PB % 4 * 8));
                        w = ok ? w : none;
                    }
                }
                const uint32_t block = c / (16 / PB);  // of the lane's channels
#pragma unroll
                for (int j = 0; j < 4; ++j) {  // token pair (2j, 2j + 1)
                    uint32_t y[2], p2[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int t = 2 * j + u, r = t & 3;  // token r of its run
                        y[u] = x.v[t];
                        // the power's byte, from bit `at`, to bits 23 to 30
                        const uint32_t at = 8 * ((r * PB & 3) + block), w = x.vp[t >> 2][r * PB / 4];
                        p2[u] = __builtin_amdgcn_alignbit(w, w, at + 9 & 31);
                    }
                    const auto pair = [&](auto which) {
                        constexpr int B = decltype(which)::value;
                        const uint32_t a = widen_fp4<B>(y[0], p2[0]), d = widen_fp4<B>(y[1], p2[1]);
                        vf[2 * B][j] = __builtin_amdgcn_perm(d, a, 0x05040100u);
                        vf[2 * B + 1][j] = __builtin_amdgcn_perm(d, a, 0x07060302u);
                    };
                    pair(std::integral_constant<int, 0>{});
                    pair(std::integral_constant<int, 1>{});
                    if constexpr (NC == 8) {
                        pair(std::integral_constant<int, 2>{});
                        pair(std::integral_constant<int, 3>{});
                    }
                }
            } else {
                if (PART) {
                    // rows behind the end may hold anything: NaN times a weight of 0 would stay
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const bool ok = counts(t0, j);
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
            if (!RING && !LAST && t0 + kBlock < stop) load(t0 + kBlock, it + 1, x);

            // many new tokens: which of the lane's 8 tokens a row sees
            uint32_t sight[MANY ? RT : 1];
            const auto row_sees = [&](int rt, int j) { return (sight[MANY ? rt : 0] >> j & 1) != 0; };
            if (MANY && PART) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    uint32_t bits = 0;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int32_t t = (int32_t)(real(t0 + 16 * i) + 4 * g);
                        Sight z;
                        z.past = pos[MANY ? rt : 0] - t;
                        z.left = src.window ? z.past - (int32_t)src.window : -0x7FFFFFFF;
                        z.sunk_to = src.window ? (int32_t)src.sinks - t : 0;
#pragma unroll
                        for (int j = 0; j < 4; ++j) bits |= z(j) ? 1u << (4 * i + j) : 0u;
                    }
                    sight[MANY ? rt : 0] = bits;
                }
            }
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
                if (PART) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[rt][j] = (MANY ? row_sees(rt, j) : counts(t0, j)) ? y[rt][j] : kNegInf;
                }
                top[rt] = y[rt][0];
#pragma unroll
                for (int j = 1; j < 8; ++j) top[rt] = fmaxf(top[rt], y[rt][j]);
                move |= top[rt] > m[rt] + kSlack;
            }
            float big[RE];
            if (HALF) {
#pragma unroll
                for (int e = 0; e < RE; ++e) {
                    big[e] = 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) big[e] = fmaxf(big[e], MANY && PART && !row_sees(e, j) ? 0.0f : vs[j]);
                    move |= big[e] >= elimit[e];
                }
            }
            if (__ballot(move) != 0) {
                const auto larger = [](float a, float b) { return fmaxf(a, b); };
                float shrink[RE];
#pragma unroll
                for (int i = 0; i < RE; ++i) {
                    shrink[i] = 1.0f;
                    if (HALF) {
                        big[i] = over_groups(big[i], larger);
                        const int e = __builtin_amdgcn_frexp_expf(big[i]), ne = big[i] >= elimit[i] ? e : E[i];
                        shrink[i] = __builtin_amdgcn_ldexpf(1.0f, E[i] - ne);
                        E[i] = ne;
                        elimit[i] = __builtin_amdgcn_ldexpf(1.0f, ne);
                        wmul[i] = __builtin_amdgcn_ldexpf(1.0f, kWeightExp - ne);
                    }
                }
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const float nm = fmaxf(m[rt], over_groups(top[rt], larger));
                    const float a = nm == kNegInf ? 1.0f : exp2_fast(m[rt] - nm);
                    m[rt] = nm;
                    mu[rt] = nm == kNegInf ? 0.0f : nm;
                    l[rt] *= a;
#pragma unroll
                    for (int n = 0; n < NC; ++n) o[rt][n] *= a * shrink[MANY ? rt : 0];
                }
            }
            if (HALF && !MANY) {
#pragma unroll
                for (int j = 0; j < 8; ++j) vs[j] *= wmul[0];
            }
            if constexpr (MANY && !HALF) {
                // a value that is not finite, seen by some rows and not by others: what it reaches is NaN, by a product of
                // what is not finite with who sees it, and it becomes 0, which a weight of 0 leaves at 0
                uint32_t bad = 0;
                if (PART) {
#pragma unroll
                    for (int n = 0; n < NC; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) bad |= infinite(vf[n][j]);
                }
                if (__builtin_expect(PART && __ballot(bad != 0) != 0, 0)) {
                    u32x4 who[RT];
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            who[rt][j] = ((sight[MANY ? rt : 0] >> 2 * j & 1) | (sight[MANY ? rt : 0] >> (2 * j + 1) & 1) << 16) * 0x3F80u;
#pragma unroll
                    for (int n = 0; n < NC; ++n) {
                        u32x4 what;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t z = vf[n][j];
                            asm("" : "+v"(z));  // (found again here: kept, it would take 32 registers)
                            const uint32_t ones = infinite(z) >> 15;
                            what[j] = ones * 0x3F80u;
                            vf[n][j] = z & ~(ones * 0xFFFFu);
                        }
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt) {
                            const f32x4 hit = mfma_bf16(what, who[rt], f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
                            for (int r = 0; r < 4; ++r) o[rt][n][r] = hit[r] > 0.0f ? __builtin_nanf("") : o[rt][n][r];
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                float w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float e = exp2_fast(y[rt][j] - mu[rt]);
                    // by the token, not by its logit: -inf * 0 has no sign
                    if (PART && !WIN) e = counts(t0, j) ? e : 0.0f;
                    l[rt] += e;
                    w[j] = !HALF ? e : MANY ? e * (vs[j] * wmul[MANY ? rt : 0]) : e * vs[j];
                    if (HALF && MANY && PART) w[j] = row_sees(rt, j) ? w[j] : 0.0f;  // (a step of NaN)
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
                load_first(base);
            }
            const uint32_t stop = FMT == kFmtPool || end - base <= kPageRun ? end : base + kPageRun;
            uint32_t it = 0, t0 = base + wave * kTile;
            if (WIN) {
                // tiles that all rows see the whole of lie side by side, others before and behind them
                const uint32_t full = all_to < stop ? all_to : stop, masked = all_from < stop ? all_from : stop;
                for (; t0 < masked; t0 += kBlock, ++it) tile(std::true_type{}, t0, stop, it, x);
                for (; t0 + kTile <= full; t0 += kBlock, ++it) tile(std::false_type{}, t0, stop, it, x);
                for (; t0 < stop; t0 += kBlock, ++it) tile(std::true_type{}, t0, stop, it, x);
            } else {
                for (; t0 + kTile <= stop; t0 += kBlock, ++it) tile(std::false_type{}, t0, stop, it, x);
                if (t0 < stop) tile(std::true_type{}, t0, stop, it, x);
            }
            if (FMT == kFmtPool) break;
        }
        if (FMT == kFmtPool && !header) {
            if (threadIdx.x == 0 && p.status) atomicOr(p.status, kDevBadHeader);
            return;
        }

        // ---- join the waves: m and l first, then the sums
        const bool whole = take == nb;
        const uint32_t slot = whole ? (src.whole ? 0 : 2 * src.W) + (uint32_t)unit : off ? 2 * w : 2 * w + 1;
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
            src.info[unit] = make_uint2(slot, parts);
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
            if (HALF) a *= __builtin_amdgcn_ldexpf(1.0f, E[MANY ? rt : 0] - kWeightExp);
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
            if (r < rows) {
                if (whole && p.direct) {
                    uint32_t seq, qh;
                    place_of(r, seq, qh);
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

template <int FMT, int D, int RT, int MODE>
__global__ __launch_bounds__(kWaves* kWave, waves_per_simd(D, RT)) void attend_kernel(Common p, Source src) {
    fetch_arguments<sizeof(Common) + sizeof(Source)>();
    __shared__ Shared<FMT, D, RT, MODE> sh;
    attend_share<FMT, D, RT, MODE>(p, src, blockIdx.x, sh);
}

// A pool's workgroups and those of the tails behind it, in one launch.
template <int FMT, int D, int RT>
__global__ __launch_bounds__(kWaves* kWave, waves_per_simd(D, RT)) void attend_both_kernel(Common p, Source pool,
                                                                                           Source tail) {
    fetch_arguments<sizeof(Common) + 2 * sizeof(Source)>();
    __shared__ union {
        Shared<kFmtPool, D, RT, kOneSeesAll> a;
        Shared<FMT, D, 1, kOneSeesAll> b;
    } sh;
    if (blockIdx.x < pool.W)
        attend_share<kFmtPool, D, RT, kOneSeesAll>(p, pool, blockIdx.x, sh.a);
    else
        attend_share<FMT, D, 1, kOneSeesAll>(p, tail, blockIdx.x - pool.W, sh.b);
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

template <int D, int V, bool MANY>
__global__ __launch_bounds__(kBlockThreads) void attend_join_kernel(JoinParams p) {
    fetch_arguments<sizeof(JoinParams)>();
    constexpr int C = D / 64, U = 8;
    constexpr int RPB = kBlockThreads / kWave / V;  // rows of a workgroup
    typedef float vec __attribute__((ext_vector_type(C)));
    const uint32_t lane = lane_id();
    const uint32_t wave = wave_uniform(threadIdx.x / kWave), w = wave % V;
    const uint32_t row = blockIdx.x * RPB + wave / V;
    if (row >= (MANY ? p.src[0].tokens : p.c.n) * p.c.Hq) return;
    const uint32_t seq = row / p.c.Hq, qh = row % p.c.Hq;  // many new tokens: `seq` is a token
    const uint32_t h = qh / p.c.group;
    uint32_t i = qh % p.c.group, row_blocks = p.src[0].row_blocks;
    uint64_t unit0 = 0;
    if constexpr (MANY) {
        // the last sequence that starts at or before the token: of 64 that are evenly apart, then of those between two
        uint32_t b = 0, range = p.c.n;
        while (range > 1) {
            const uint32_t each = (range + kWave - 1) / kWave, at = b + lane * each;
            const bool before = lane * each < range && p.src[0].starts[at] <= (int32_t)seq;
            const uint32_t k = __builtin_popcountll(__ballot(before));
            if (k == 0) return;
            b += (k - 1) * each;
            range = (k - 1) * each + each < range ? each : range - (k - 1) * each;
        }
        const Fresh x = fresh_of(p.src[0], b);
        if (seq - x.first >= x.count) return;  // of no sequence
        i += (seq - x.first) * p.c.group;
        unit0 = p.rt[0] == 1 ? first_unit<1>(b, x.first, p.c.group, p.c.H) : first_unit<2>(b, x.first, p.c.group, p.c.H);
        row_blocks = p.rt[0] == 1 ? row_blocks_of<1>(x.count, p.c.group) : row_blocks_of<2>(x.count, p.c.group);
    }
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
        if (MANY) {
            // (where starts were wrong no workgroup wrote it, and it may hold anything)
            const u32x2 z = scalar_load<u32x2>(x.info + unit0 + h * row_blocks + r / tile);
            const bool ok = (z.x < 2 * x.W) & (z.y <= x.W) & (z.x + 2 * z.y <= 2 * x.W + 2);
            info[s] = u32x2{ok ? z.x : 0, ok ? z.y : 0};
        } else {
            info[s] = scalar_load<u32x2>(x.info + (x.pool ? 0 : seq * p.c.H * x.row_blocks) + h * x.row_blocks + r / tile);
        }
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
    // with one, us: pool of 15 agents, 60 rows, heads of 128: 131071 tokens 81 and 110, 4096 with tails 15.1 and 18.2,
    // 1024 12.3 and 10.0. Pages, 8 sequences of 8192, 2 kv heads: heads of 64, 17 rows int8 13.0 and 14.1, bf16 13.9 and
    // 16.5; heads of 128, 32 rows int8 19.4 and 17.5, bf16 21.1 and 19.2, 33 rows 21.0 and 25.4, 21.4 and 36.6. Not taken
    // yet: two tiles for 17 to 32 rows of heads of 128 in larger calls (15 sequences of 4096, 8 kv heads, 17 rows: int8 38.0
    // and 48.5, bf16 56.0 and 80.8; 32 rows: 40.7 and 49.8, 58.0 and 81.8).
    const uint64_t most_blocks = (max_tokens + kBlock - 1) / kBlock;
    const bool enough = units_of_rows * ((rows + 31) / 32) * most_blocks >= 256ull * waves_per_simd(d, 2);
    return plan_of(units_of_rows, rows, max_tokens, d, rows > one_tile && enough ? 2 : 1, direct);
}

template <int FMT, int D, int MODE>
hipError_t launch_pages(uint32_t rt, uint32_t grid, const Common& p, const Source& s, hipStream_t stream) {
    return launch_kernel(rt == 1 ? attend_kernel<FMT, D, 1, MODE> : attend_kernel<FMT, D, 2, MODE>, dim3(grid),
                         dim3(kWaves * kWave), stream, p, s);
}
template <int D, int MODE>
hipError_t launch_pages_as(uint32_t format, uint32_t rt, uint32_t grid, const Common& p, const Source& s,
                           hipStream_t stream) {
    switch (format) {
        case kPageBf16: return launch_pages<kFmtBf16, D, MODE>(rt, grid, p, s, stream);
        case kPageInt8: return launch_pages<kFmtInt8, D, MODE>(rt, grid, p, s, stream);
        case kPageFp8: return launch_pages<kFmtFp8, D, MODE>(rt, grid, p, s, stream);
        default: return launch_pages<kFmtFp4, D, MODE>(rt, grid, p, s, stream);
    }
}
template <int D>
hipError_t launch_pages_of(int mode, uint32_t format, uint32_t rt, uint32_t grid, const Common& p, const Source& s,
                           hipStream_t stream) {
    return mode == kMany        ? launch_pages_as<D, kMany>(format, rt, grid, p, s, stream)
           : mode == kOneWindow ? launch_pages_as<D, kOneWindow>(format, rt, grid, p, s, stream)
                                : launch_pages_as<D, kOneSeesAll>(format, rt, grid, p, s, stream);
}
template <int FMT, int D>
hipError_t launch_both(uint32_t rt, uint32_t grid, const Common& p, const Source& a, const Source& b, hipStream_t stream) {
    return launch_kernel(rt == 1 ? attend_both_kernel<FMT, D, 1> : attend_both_kernel<FMT, D, 2>, dim3(grid),
                         dim3(kWaves * kWave), stream, p, a, b);
}
template <int D>
hipError_t launch_both_of(uint32_t format, uint32_t rt, uint32_t grid, const Common& p, const Source& a, const Source& b,
                          hipStream_t stream) {
    switch (format) {
        case kPageBf16: return launch_both<kFmtBf16, D>(rt, grid, p, a, b, stream);
        case kPageInt8: return launch_both<kFmtInt8, D>(rt, grid, p, a, b, stream);
        case kPageFp8: return launch_both<kFmtFp8, D>(rt, grid, p, a, b, stream);
        default: return launch_both<kFmtFp4, D>(rt, grid, p, a, b, stream);
    }
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

// Many new tokens: up to 32 rows of a sequence and kv head (its new tokens times the heads that share it) a unit. Two row
// tiles from 17 rows in the mean on: 15 sequences with drafts behind 8192 tokens, 8 kv heads, with two and with one, us:
// heads of 128, 20 rows e4m3 66.6 and 85.9, bf16 104 and 151, 16 rows 65.2 and 60.3, 103 and 101; heads of 64, 20 rows
// 39.4 and 50.1, 57.2 and 79.8, 16 rows 38.4 and 35.2, 56.0 and 54.0.
AttendPlan many_attend_plan(uint32_t n_seqs, uint32_t n_tokens, uint32_t H, uint32_t Hq, uint32_t d, uint64_t max_tokens,
                            uint32_t window, uint32_t sinks) {
    AttendPlan a{};
    const uint64_t rows = (uint64_t)n_tokens * (Hq / H);
    a.rt = rows > 16ull * n_seqs ? 2 : 1;
    a.row_blocks = 1;
    a.units = (rows / (16 * a.rt) + n_seqs) * H;  // at most
    // (a sequence's rows see the tokens of one row, and with a window as many more as it has new ones)
    const uint64_t seen = window ? seen_tokens(max_tokens, (uint64_t)window + n_tokens, sinks) : max_tokens;
    a.blocks = a.units * ((seen + kBlock - 1) / kBlock);
    const uint64_t places = 256ull * waves_per_simd(d, a.rt);
    a.W = a.blocks / kMinBlocks < places ? a.blocks / kMinBlocks : places;
    if (a.W < 1) a.W = 1;
    a.slots = 2 * a.W;
    a.room = a.bytes(d);
    return a;
}

uint64_t many_attend_room(uint32_t n_seqs, uint64_t rows, uint32_t H, uint32_t d, uint64_t max_tokens) {
    const uint64_t units = (rows / 16 + n_seqs) * H, places = 256ull * waves_per_simd(d, 1);
    uint64_t w = units * ((max_tokens + kBlock - 1) / kBlock) / kMinBlocks;
    w = w < 1 ? 1 : w < places ? w : places;
    return align_up(2 * w * 32 * (d + 2) * 4 + units * 8, 256);
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
        const uint64_t most = (uint64_t)a.tail.table_cols * lay.P;
        page_plan = a.starts ? many_attend_plan(a.n, a.tokens, a.H, a.Hq, a.d, most, a.tail.window, a.tail.sinks)
                             : page_attend_plan(a.n, a.H, a.Hq, a.d, seen_tokens(most, a.tail.window, a.tail.sinks), has_pool);
        ws += place_source(pages, page_plan, a.d, ws);
        pages.pages = a.tail.pages;
        pages.table = a.tail.table;
        pages.table_stride = a.tail.table_stride;
        pages.lens = a.tail.lens;
        pages.window = a.tail.window;
        pages.sinks = a.tail.sinks;
        if (a.starts) {
            pages.starts = a.starts;
            pages.tokens = a.tokens;
        }
        pages.table_cols = a.tail.table_cols;
        pages.num_pages = lay.num_pages;
        pages.page_shift = 31 - __builtin_clz(lay.P);
        pages.page_bytes = lay.page_bytes;
        pages.steps = lay.steps;
    }
    hipError_t e;
    if (has_pool && has_pages) {
        const uint32_t grid = pool.W + pages.W;
        e = a.d == 64 ? launch_both_of<64>(a.tail.lay.format, pool_plan.rt, grid, p, pool, pages, stream)
                      : launch_both_of<128>(a.tail.lay.format, pool_plan.rt, grid, p, pool, pages, stream);
    } else if (has_pool) {
        e = a.d == 64 ? launch_pages<kFmtPool, 64, kOneSeesAll>(pool_plan.rt, pool.W, p, pool, stream)
                      : launch_pages<kFmtPool, 128, kOneSeesAll>(pool_plan.rt, pool.W, p, pool, stream);
    } else {
        const uint32_t format = a.tail.lay.format;
        const int mode = a.starts ? kMany : a.tail.window ? kOneWindow : kOneSeesAll;
        e = a.d == 64 ? launch_pages_of<64>(mode, format, page_plan.rt, pages.W, p, pages, stream)
                      : launch_pages_of<128>(mode, format, page_plan.rt, pages.W, p, pages, stream);
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
    const uint64_t rows = (uint64_t)(a.starts ? a.tokens : a.n) * a.Hq;
    // One wave joins a row of few parts, four one of many. A call with one and with four, us: pages of 1, 4, 8, 15
    // and 32 sequences of 4096 tokens (W / units 64, 16, 8, 4, 2) 10.4 and 10.0, 13.4 and 13.1, 18.3 and 18.6, 28.8
    // and 29.2, 48.0 and 48.7; a pool of 8192 tokens for 4 agents (32) 12.2 and 10.7, of 131071 over 2 kv heads (256) 32.9
    // and 19.9. It goes by the mean: of 100 sequences (5) one of 40000 tokens among 99 of 100 takes 31.2, with four 16.4.
    const bool few = first.whole || first.W <= 6 * first.units;
    const dim3 grid((uint32_t)(few ? (rows + 3) / 4 : rows));
    const auto join = [&](auto one, auto four) { return launch_kernel(few ? one : four, grid, dim3(kBlockThreads), stream, j); };
    if (a.starts)
        return a.d == 64 ? join(attend_join_kernel<64, 1, true>, attend_join_kernel<64, 4, true>)
                         : join(attend_join_kernel<128, 1, true>, attend_join_kernel<128, 4, true>);
    return a.d == 64 ? join(attend_join_kernel<64, 1, false>, attend_join_kernel<64, 4, false>)
                     : join(attend_join_kernel<128, 1, false>, attend_join_kernel<128, 4, false>);
}

}  // namespace kvc
