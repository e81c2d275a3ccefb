// prompt_kernels.hip - attention of many new tokens of each sequence over its
// pages (a prompt, a part of one), for gfx950.
//
// The query rows of a sequence and kv head are its new tokens times the query heads
// that share the kv head, token by token. A workgroup takes a block of 128 of them, 32 a
// wave, and walks the tokens that they see in tiles of 32, with one pass over the data
// (running maximum m and sum l):
//     S^T = K Q^T           32x32x16 matrix instructions, tokens x rows
//     p = exp2(f S - m)     in the lanes that hold S
//     O^T += V^T p^T        32x32x16, channels x rows
// In both products a lane's column is one query row (lane % 32), shared with lane + 32,
// so m and l are its own registers. S^T leaves a lane with tokens 8j + 4 (lane / 32) +
// 0..3, and the second product takes its tokens in that order: the transposed LDS read
// gives four tokens of one channel to a lane, so V stays in LDS as it is in memory.
//
// What bounds it: matrix and vector instructions. A tile of a wave costs 16 products of 32
// cycles (heads of 128) and some 250 cycles of exponentials, sums and packing for two
// waves each, so products have to run beside softmax all the time: a turn has the next tile's keys, this one's
// weights and the values of the one before, which are independent, two products beside two weights. Keys and
// values lie in a ring of four tiles in LDS, filled by loads that nothing waits for but the end of
// two tiles (bf16), or widened on their way (8 bits: binary16, where codes are exact; 4 bits: bf16, the same). One prompt of 8192
// tokens (8 kv heads of 128, 4 heads each): bf16 541 to 573 us from card to card and by what runs beside it, 960 to 1016
// TFLOP/s of what the mask leaves, of a SIMD's cycles the matrix core 53 %, the VALU 52 %, at 1.9 GHz: the clock falls as
// power allows (a build with 12 % more cycles took 1 % longer). Back to back on a card where bf16 takes 572: e4m3 722, int8
// 745, 4 bits 590 us: steps of 8 bits cost a product each for logits and weights, and codes their widening. Heads of 64, with
// as many exponentials for half the products: 333 us. Vector registers spilled: where tiles are shared out 23 (e4m3) and 24
// (int8), with heads of 64 38, 50, 23 (4 bits) and 9 (bf16); where not, with heads of 64, 18, 20, 2 and 0.
// Measured and left out: tiles of 64 tokens (7 to 20 % longer), 256 rows a
// workgroup, operands asked for four products ahead.
//
// Weights are rounded once: to bf16 (2^-8: a row sums over many tokens, and these errors do not add up as the
// weights do), or, times their step and a power of two of the row, to binary16 (2^-11). m moves when a tile's maximum
// passes it by kSlack, so most tiles need no exchange between lanes and no rescaling.
#include "attend.h"
#include "kernels_common.h"
#include "lds_fetch.h"
#include "page_codes.h"

#include <type_traits>

namespace kvc {
namespace {

constexpr int kDevBadPage = 32, kDevBadLength = 64, kDevBadStart = 128;  // KVC_DEV_*
constexpr uint32_t kTokens = 32;   // of a tile
constexpr uint32_t kRows = 128;    // of a block, 32 a wave
constexpr int kWaves = 4;
constexpr uint32_t kRun = 16;      // tokens that lie in one page: a wave fetches a run of each two tiles
constexpr float kSlack = 3.0f;     // m moves when a tile's maximum passes it by this (powers of two)
constexpr int kWeightExp = 12;     // binary16 weights: the largest stays below 2^(12 + 3 + 1)
constexpr uint32_t kMinShare = 16;  // tiles of a share, at least
constexpr uint32_t kCus = 256;
constexpr uint32_t workgroups(uint32_t d) { return d == 64 ? 3 : 2; }  // of a CU: registers bound them
constexpr uint32_t kBegin = 8;      // to begin and end a block takes as long as so many tiles
constexpr float kNegInf = -__builtin_inff();
constexpr bool half_products(int fmt) { return fmt == kPageInt8 || fmt == kPageFp8; }

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

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
    uint32_t shares;  // of the tiles of a kv head, one a workgroup (0: a block a workgroup, none is cut up)
    float scale_log2;
    float* part;  // of a share's part of a block that is cut up: sums, as lanes hold them, then {m, l} of each row
    uint2* info;  // of each block: its first share and its parts, 0 where it is not cut up
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

// LDS: tile j of keys, and of values, is in buffer (j - the share's first) % 4. The steps of both (8 bits) come with the keys and are read
// for as long as the values, so they have eight places.
template <int FMT, int D>
struct Tiles {
    static constexpr uint32_t kBytes = kTokens * D * 2;
    alignas(16) uint8_t kv[2][4][kBytes];  // [keys, values][buffer]
    float steps[half_products(FMT) ? 2 : 1][8][half_products(FMT) ? kTokens : 1];
    float big[8][2];  // largest step of the values of each run (8 bits)
    uint32_t odd[8];  // a tile's values or their steps are not all finite: 1 + the tile
};

// Tiles of what a block's rows see, from its first row's position to its last's: tokens below `sunk` and from `lo` to `end`.
struct Range {
    uint32_t sunk, lo, end;
    uint32_t tiles0, from, tiles;  // tiles of the sinks; the first behind them; all
};
__device__ __forceinline__ Range range_of(const PromptParams& p, int32_t pos_lo, int32_t pos_hi) {
    Range r;
    r.end = pos_hi < 0 ? 0 : pos_hi + 1;
    r.lo = p.window && pos_lo >= 0 && (uint32_t)pos_lo >= p.window ? pos_lo - p.window + 1 : 0;
    r.sunk = p.sinks < r.lo ? p.sinks : r.lo;
    r.tiles0 = (r.sunk + kTokens - 1) / kTokens;
    r.from = r.lo / kTokens > r.tiles0 ? r.lo / kTokens : r.tiles0;
    const uint32_t last = (r.end + kTokens - 1) / kTokens;
    r.tiles = r.tiles0 + (last > r.from ? last - r.from : 0);
    return r;
}

// A sequence's new tokens and length. Sequences are taken from the last to the first (`i` counts them so), and a
// sequence's blocks too, so that the longest of a prompt come first.
struct Sequence {
    uint32_t b, first, m;  // first: its first row (~0: its starts are wrong)
    int32_t len;
    uint32_t blocks;
    __device__ __forceinline__ int32_t pos_of(uint32_t row, uint32_t group) const { return len - (int32_t)m + (int32_t)(row / group); }
};
template <bool REPORT>
__device__ __forceinline__ Sequence sequence_at(const PromptParams& p, uint32_t i) {
    Sequence s{};
    if (i >= p.n) return s;
    s.b = p.n - 1 - i;
    const int32_t a = p.starts[s.b], e = p.starts[s.b + 1], given = p.lens[s.b];
    const bool bad = a < 0 || e < a || (uint32_t)e > p.rows;
    const uint32_t most = p.table_cols << p.page_shift;
    s.len = given < 0 ? 0 : (uint32_t)given > most ? (int32_t)most : given;
    if (REPORT && p.status && (bad || s.len != given))
        atomicOr(p.status, (bad ? kDevBadStart : 0) | (s.len != given ? kDevBadLength : 0));
    s.first = bad ? ~0u : (uint32_t)a;
    s.m = bad ? 0 : e - a;
    s.blocks = (s.m * p.group + kRows - 1) / kRows;
    return s;
}
__device__ __forceinline__ Sequence uniform(const Sequence& s, int lane) {
    const auto of = [&](uint32_t v) { return (uint32_t)__builtin_amdgcn_readlane(v, lane); };
    return Sequence{of(s.b), of(s.first), of(s.m), (int32_t)of(s.len), of(s.blocks)};
}
__device__ __forceinline__ uint64_t uniform(uint64_t x) { return (uint64_t)wave_uniform((uint32_t)(x >> 32)) << 32 | wave_uniform((uint32_t)x); }
// Tiles that a block sees; one that sees none has an empty one, so that its rows are written.
__device__ __forceinline__ uint32_t tiles_of(const PromptParams& p, const Sequence& s, uint32_t block) {
    const uint32_t row0 = block * kRows, left = s.m * p.group - row0;
    const uint32_t t = range_of(p, s.pos_of(row0, p.group), s.pos_of(row0 + (left < kRows ? left : kRows) - 1, p.group)).tiles;
    return t ? t : 1;
}

// Where few blocks would leave workgroups idle, or wait for the longest, all tiles of a kv head are shared out evenly: the
// blocks stand in a row, and each workgroup takes as many tiles as the others, from where the one before it ends. What
// blocks of a sequence see grows evenly, so the row has the last with the first, the last but one with the second, ...:
// each such pair counts as long as the first pair is (the one in the middle, of an odd number, half as long; with what
// it takes to begin a block), and how far into a pair a share begins or ends is taken in proportion.
struct Pairs {
    uint32_t len, last;  // of a pair, and of the last one
    uint64_t all;        // of all
};
__device__ __forceinline__ Pairs pairs_of(const PromptParams& p, const Sequence& s) {
    Pairs x{};
    if (s.blocks == 0) return x;
    x.len = tiles_of(p, s, 0) + tiles_of(p, s, s.blocks - 1) + 2 * kBegin;
    x.last = s.blocks % 2 ? (x.len + 1) / 2 : x.len;
    x.all = (uint64_t)((s.blocks - 1) / 2) * x.len + x.last;
    return x;
}
// A pair's blocks and their tiles (`low` of a middle one: none).
struct Pair {
    uint32_t high, low, tiles_high, tiles_low, len;
    // tiles up to `at` of the pair's length
    __device__ __forceinline__ uint32_t tiles_to(uint32_t at) const {
        uint64_t q;
        uint32_t r;
        divmod_u64((uint64_t)at * (tiles_high + tiles_low), len, q, r);
        return (uint32_t)q;
    }
};
__device__ __forceinline__ Pair pair_at(const PromptParams& p, const Sequence& s, const Pairs& x, uint32_t q) {
    Pair r;
    r.high = s.blocks - 1 - q;
    r.low = q;
    r.tiles_high = tiles_of(p, s, r.high);
    r.tiles_low = r.low < r.high ? tiles_of(p, s, r.low) : 0;
    r.len = q == (s.blocks - 1) / 2 ? x.last : x.len;
    return r;
}

// Over the wave's lanes up to this one, of numbers below 2^50.
__device__ __forceinline__ uint64_t scan_lanes64(uint64_t v) {
    return scan_lanes((uint32_t)v & 0xFFFFF) + ((uint64_t)scan_lanes((uint32_t)(v >> 20)) << 20);
}
__device__ __forceinline__ uint64_t read_lane64(uint64_t v, int lane) {
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((uint32_t)(v >> 32), lane) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((uint32_t)v, lane);
}
// The first sequence with which the sum of `of` passes `at`, and the sums before it: a wave finds it, a lane a sequence.
// `at` comes from the sum of all, which is known at once where the lanes hold every sequence. Where starts are wrong
// there is none: rows could be given many times over.
struct Found {
    bool any;
    Sequence s;
    uint32_t i;
    uint64_t at, before;
};
template <class F, class A>
__device__ __forceinline__ Found find_sequence(const PromptParams& p, F of, A place) {
    uint64_t all = 0, mine = 0, up = 0;
    bool bad = false;
    Sequence s{};
    for (uint32_t base = 0; base < p.n; base += kWave) {
        s = sequence_at<true>(p, base + lane_id());
        bad |= s.first == ~0u;
        mine = of(s);
        up = scan_lanes64(mine);
        all += read_lane64(up, 63);
    }
    if (__ballot(bad) != 0) all = 0;
    const uint64_t at = place(all);
    if (at >= all) return Found{};
    uint64_t before = 0;
    for (uint32_t base = 0;; base += kWave) {
        if (p.n > kWave) {
            s = sequence_at<false>(p, base + lane_id());
            mine = of(s);
            up = scan_lanes64(mine);
        }
        const uint64_t these = read_lane64(up, 63);
        if (at < before + these) {
            const int l = __builtin_popcountll(__ballot(before + up <= at));
            return Found{true, uniform(s, l), base + l, at, before + read_lane64(up - mine, l)};
        }
        before += these;
    }
}
// Where share k of `count` begins in `all` tiles. A CU's first workgroup goes before its second, which goes before its
// third (a SIMD takes its oldest wave first), so that with equal shares the later ones end by themselves: four chunked
// prompts, int8, shares of 76 tiles, after 136 and 158 us. Long shares are given out in that order, in proportions of 18
// to 16 to 14 (the call with bf16 pages 123 -> 116 us); short ones are equal, as are then most blocks or their halves,
// of which fewer are cut up (one prompt of 2000 tokens, shares of 39 tiles: 64 us, in those proportions 72).
constexpr uint32_t kLongShare = 64;
struct Bounds {
    uint64_t all;
    uint32_t count, row;  // row: shares of a kv head with which each CU has one workgroup
    uint32_t less;        // of 18, with each further workgroup of a CU
    __device__ __forceinline__ uint32_t weight_to(uint32_t k) const {
        return 18 * k - less * ((k > row ? k - row : 0) + (k > 2 * row ? k - 2 * row : 0));
    }
    __device__ __forceinline__ uint64_t operator()(uint32_t k) const {
        if (k >= count) return all;
        uint64_t q;
        uint32_t r;
        if (less == 0) {
            divmod_u64(all + count - 1, count, q, r);
            return q * k < all ? q * k : all;
        }
        divmod_u64(all * weight_to(k), weight_to(count), q, r);
        return q;
    }
};
__device__ __forceinline__ Bounds bounds_of(const PromptParams& p, uint64_t all) {
    const uint64_t most = all / kMinShare;
    const uint32_t count = most < 1 ? 1 : most < p.shares ? (uint32_t)most : p.shares;
    return Bounds{all, count, kCus / p.H ? kCus / p.H : 1, all >= (uint64_t)kLongShare * count ? 2u : 0u};
}
// A block's place in the list of all (those of the sequences before it, rounded up one by one, are no more).
__device__ __forceinline__ uint32_t first_block(const PromptParams& p, uint32_t b, uint32_t first) { return first * p.group / kRows + b; }
// The last sequence whose blocks' places begin at or before this one: of 64 that are evenly apart, then of those between
// two. (n: none. Wrong starts give some sequence, or none.)
__device__ __forceinline__ uint32_t sequence_of(const PromptParams& p, uint32_t place) {
    uint32_t b = 0, range = p.n;
    for (;;) {
        const uint32_t each = (range + kWave - 1) / kWave, at = lane_id() * each;
        const bool before = at < range && first_block(p, b + at, p.starts[b + at]) <= place;
        const uint32_t k = __builtin_popcountll(__ballot(before));
        if (k == 0) return p.n;
        b += (k - 1) * each;
        range = range - (k - 1) * each < each ? range - (k - 1) * each : each;
        if (range <= 1) return b;
    }
}

// SHARED: the tiles of all blocks are shared out.
template <int FMT, int D, bool SHARED>
__global__ __launch_bounds__(kWaves* kWave, workgroups(D)) void prompt_kernel(PromptParams p) {
    fetch_arguments<sizeof(PromptParams)>();
    constexpr bool HALF = half_products(FMT);
    constexpr int KS = D / 16, CB = D / 32;  // steps of a key product, blocks of channels
    __shared__ Tiles<FMT, D> sh;
    const uint32_t h = blockIdx.x % p.H, share = blockIdx.x / p.H;
    Sequence sq;
    Pairs pairs{};
    uint32_t index = 0, block = 0, half = 0;
    uint64_t at = 0, left = 0;  // where the share is in its sequence's row of blocks, and how much of it is left
    Bounds bounds{};
    if constexpr (SHARED) {
        const Found f = find_sequence(p, [&](const Sequence& s) { return pairs_of(p, s).all; }, [&](uint64_t all) {
            bounds = bounds_of(p, all);
            const uint64_t x0 = bounds(share);
            left = bounds(share + 1) - x0;
            return x0;
        });
        if (!f.any) return;
        sq = f.s;
        index = f.i;
        at = f.at - f.before;
        pairs = pairs_of(p, sq);
    } else if (p.n > kWave) {
        // by places: with all sequences counted by each workgroup, a call of 16384 sequences of one token (8 kv heads) takes 30
        // ms, by places 2.4, and the former grows with their square. There are as many places as sequences at least, so each
        // sequence is looked at for what is wrong with it.
        if (h == 0 && share < p.n) (void)sequence_at<true>(p, share);
        const uint32_t place = p.rows * p.group / kRows + p.n - 1 - share, b = sequence_of(p, place);
        if (b >= p.n) return;
        sq = uniform(sequence_at<false>(p, p.n - 1 - b), 0);
        block = place - first_block(p, b, sq.first);
        if (block >= sq.blocks) return;
    } else {
        const Found f = find_sequence(p, [](const Sequence& s) { return (uint64_t)s.blocks; }, [&](uint64_t) { return share; });
        if (!f.any) return;
        sq = f.s;
        block = f.s.blocks - 1 - (share - (uint32_t)f.before);
    }
    for (bool again = false;; again = true) {
    if constexpr (SHARED) {
        // the same in all lanes, which the compiler does not see (20 vector registers)
        at = uniform(at);
        left = uniform(left);
        bounds = Bounds{uniform(bounds.all), wave_uniform(bounds.count), bounds.row, wave_uniform(bounds.less)};
        pairs = Pairs{wave_uniform(pairs.len), wave_uniform(pairs.last), uniform(pairs.all)};
        sq = uniform(sq, 0);
        index = wave_uniform(index);
        half = wave_uniform(half);
    }
    uint32_t part0 = 0, part1 = 0xFFFFFFFFu;  // tiles of the block, of
    uint32_t tiles = 0;
    if constexpr (SHARED) {
        if (left == 0) return;
        if (at == pairs.all) {
            do sq = uniform(sequence_at<false>(p, ++index), 0);
            while (sq.blocks == 0);
            pairs = pairs_of(p, sq);
            at = 0;
        }
        uint64_t q;
        uint32_t a;
        divmod_u64(at, pairs.len, q, a);
        const Pair x = pair_at(p, sq, pairs, (uint32_t)q);
        const uint32_t e = x.len - a < left ? x.len : a + (uint32_t)left, from = x.tiles_to(a), to = x.tiles_to(e);
        if (half == 0) {
            block = x.high;
            tiles = x.tiles_high;
            part0 = from < tiles ? from : tiles;
            part1 = to < tiles ? to : tiles;
        } else {
            block = x.low;
            tiles = x.tiles_low;
            part0 = from > x.tiles_high ? from - x.tiles_high : 0;
            part1 = to > x.tiles_high ? to - x.tiles_high : 0;
        }
        if (part0 == 0 && part1 != 0 && threadIdx.x == 0) {
            // the share that begins a block counts the shares that go on with it
            const uint32_t all = half ? x.tiles_high + x.tiles_low : x.tiles_high;
            uint32_t parts = part1 < tiles ? 1 : 0;
            const uint64_t mine = bounds(share + 1);  // e, in the row of all
            for (uint32_t reached = to; reached < all; ++parts) {
                const uint64_t end = e + (bounds(share + 1 + parts) - mine);
                reached = end < x.len ? x.tiles_to((uint32_t)end) : x.tiles_high + x.tiles_low;
            }
            p.info[(uint64_t)(first_block(p, sq.b, sq.first) + block) * p.H + h] = make_uint2(share, parts);
        }
        half ^= 1;
        if (half == 0) {
            at += e - a;
            left -= e - a;
        }
        if (part0 >= part1) {
            // a share too short for a tile of a block that it is inside of
            if (part0 > 0 && part0 < tiles) {
                float* to = p.part + ((uint64_t)(2 * share) * p.H + h) * (kRows * (D + 2)) + kRows * D;
                if (threadIdx.x < kRows) *reinterpret_cast<float2*>(to + 2 * threadIdx.x) = make_float2(kNegInf, 0.0f);
            }
            continue;
        }
    }
    const bool cut = SHARED && part1 - part0 < tiles;
    if (again) __syncthreads();  // the block before is out of LDS
    // (new to the compiler for each block, or it would keep whatever follows from them alone: 40 registers)
    uint32_t thread = threadIdx.x;
    asm volatile("" : "+v"(thread));
    const uint32_t lane = thread % kWave, wave = wave_uniform(thread / kWave);
    const uint32_t col = lane & 31, hi = lane >> 5;
    const uint32_t row0 = block * kRows;
    const uint32_t nrows = sq.m * p.group - row0 < kRows ? sq.m * p.group - row0 : kRows;
    const int32_t block_lo = sq.pos_of(row0, p.group);
    const Range see = range_of(p, block_lo, sq.pos_of(row0 + nrows - 1, p.group));
    const auto start_of = [&](uint32_t i) { return (i < see.tiles0 ? i : i - see.tiles0 + see.from) * kTokens; };
    const uint32_t j0 = part0, j1 = part1 < see.tiles ? part1 : see.tiles;

    // ---- this lane's row; a lane without one takes the block's last, which is not written
    const uint32_t my_row = wave * 32 + col;
    const bool has_row = my_row < nrows;
    const uint32_t R = row0 + (has_row ? my_row : nrows - 1);
    const uint32_t tok = R / p.group, qh = h * p.group + R % p.group;
    const int32_t pos = sq.pos_of(R, p.group);
    // positions of the wave's rows
    const int32_t wave_lo = __builtin_amdgcn_readlane(pos, 0), wave_hi = __builtin_amdgcn_readlane(pos, 31);

    // ---- tiles from memory: two at a time, of which a wave fetches one run of 16 tokens, from one page. Tokens that
    // no row sees may hold anything, NaN too, which times a weight of 0 would stay: a token that is seen takes their
    // place, of the run if it has one, else the last of all.
    struct Run {
        uint32_t tile, t;     // its tile, and first token
        bool any, own, whole; // there is one; it is the tile's own; all of it is seen
        const uint8_t *rows, *steps;  // its keys
    };
    const uint32_t P = 1u << p.page_shift;
    constexpr uint32_t CODE = page_code_bytes(FMT, D), STEP = page_step_bytes(FMT, D);
    const uint64_t to_values = (uint64_t)p.H * P * CODE, to_value_steps = (uint64_t)p.H * P * STEP;
    const int32_t* row_of_table = p.table + sq.b * p.table_stride;
    // tiles from `plain0` to `plain1` - 1 lie behind the sinks' and are seen whole
    const uint32_t plain0 = see.tiles0 > j0 ? see.tiles0 : j0;
    const uint32_t seen0 = (see.lo + kTokens - 1) / kTokens;  // of the sequence's tiles
    const uint32_t skip = see.from - see.tiles0;
    const uint32_t from_lo = seen0 > skip ? seen0 - skip : 0, to_end = see.end / kTokens > skip ? see.end / kTokens - skip : 0;
    const uint32_t first_plain = plain0 > from_lo ? plain0 : from_lo, end_plain = to_end < j1 ? to_end : j1;
    // this wave's run of tiles j and j + 1
    const auto run_of = [&](uint32_t j) {
        Run r{};
        r.tile = j + wave / 2;
        if (r.tile >= first_plain && r.tile < end_plain) {
            r.any = r.own = r.whole = true;
            r.t = (r.tile + skip) * kTokens + kRun * (wave % 2);
        } else {
            r.any = (int32_t)r.tile >= (int32_t)j0 && r.tile < j1;
            if (!r.any) return r;
            const uint32_t t = start_of(r.tile) + kRun * (wave % 2);
            r.own = (t < see.end) & ((t < see.sunk) | (t + kRun > see.lo));
            r.t = r.own ? t : (see.end - 1) & ~(kRun - 1);
            r.whole = r.own & (t + kRun <= see.end) & ((t + kRun <= see.sunk) | (t >= see.lo));
        }
        // (through the scalar cache: a vector load's wait would be for every tile on its way too)
        uint32_t page = *(const __attribute__((address_space(4))) uint32_t*)(uint64_t)(row_of_table + (r.t >> p.page_shift));
        if (__builtin_expect(page >= p.num_pages, 0)) {
            if (p.status && lane == 0) atomicOr(p.status, kDevBadPage);
            page = 0;
        }
        const uint32_t line = h * P + (r.t & (P - 1));
        const uint8_t* at = p.pages + (uint64_t)page * p.page_bytes;
        r.rows = at + (uint64_t)line * CODE;
        r.steps = at + p.steps + (uint64_t)line * STEP;
        return r;
    };
    // registers of tiles on their way (formats that are widened)
    constexpr int NR = FMT == kPageBf16 ? 1 : (kRun * CODE + 1023) / 1024;  // 16-byte loads of a lane
    u32x4 raw[2][NR];
    uint32_t raw_step[2];
    // (buf: the tile's buffer is known when this is compiled, see below)
    const auto ask = [&](int kv, const Run& x, uint32_t buf) __attribute__((always_inline)) {
        if (!x.any) return;
        // the row that stands for row r of a run that is not whole
        const auto other = [&](uint32_t r) {
            const uint32_t t = x.t, token = t + r;
            const uint32_t last = see.end - 1 - t, near = t < see.sunk ? see.sunk - 1 - t : see.lo - t;
            const bool hidden = (token >= see.sunk) & (token < see.lo), none = (token >= see.end) | !x.own;
            return none ? last : hidden ? near : r;
        };
        const uint8_t* rows = kv ? x.rows + to_values : x.rows;
        const uint8_t* steps = kv ? x.steps + to_value_steps : x.steps;
        if constexpr (FMT == kPageBf16) {
            constexpr int N = kRun * CODE / 1024, RPI = 1024 / CODE;  // loads, and rows of one
            uint8_t* to = sh.kv[kv][buf] + kRun * (wave % 2) * CODE;
            uint32_t off[N];
#pragma unroll
            for (uint32_t u = 0; u < (uint32_t)N; ++u) {
                // of row r the chunk whose place is at16: places change by exclusive or, so the same change leads back
                const uint32_t r = u * RPI + lane / (CODE / 16), at16 = lane % (CODE / 16);
                off[u] = kv ? place_v<D>(r, at16) : place_k<D>(r, at16);
            }
            if (!x.whole) {
#pragma unroll
                for (int u = 0; u < N; ++u) off[u] = off[u] % CODE + other(off[u] / CODE) * CODE;
            }
            // (offsets are unsigned: the base is as far below as the instructions add at most)
#pragma unroll
            for (int u = 0; u < N; ++u) off[u] += (N - 1 - u) * 1024;
            fetch16(rows - (N - 1) * 1024, off, to);
        } else if constexpr (FMT == kPageFp4) {
            const uint32_t r = x.whole ? lane / 4 : other(lane / 4);
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
                raw[kv][u] = *reinterpret_cast<const u32x4*>(
                    rows + (x.whole ? u * 1024 + lane * 16 : other((u * 1024 + lane * 16) / CODE) * CODE + lane * 16 % CODE));
            if (kv == 0) {
                const uint32_t at = (x.whole ? lane % kRun : other(lane % kRun)) * STEP;
                raw_step[0] = *reinterpret_cast<const uint32_t*>(steps + at);
                raw_step[1] = *reinterpret_cast<const uint32_t*>(steps + to_value_steps + at);
            }
        }
    };
    // Tiles that all rows from position `lo` to `hi` see the whole of: from `first` on, `count` of them. (Without those
    // among the sinks, where there is a window: they take the general way.)
    struct Whole {
        uint32_t first, count;
        __device__ __forceinline__ bool operator()(uint32_t j) const { return j - first < count; }
    };
    const auto whole_for = [&](int32_t lo, int32_t hi) {
        Whole w;
        const int32_t left = p.window ? hi - (int32_t)p.window + 1 : 0;  // the first token that row hi sees
        const uint32_t a = left > 0 ? (left + kTokens - 1) / kTokens : 0, b = lo < 0 ? 0 : (lo + 1) / kTokens;
        const uint32_t f = a > skip ? a - skip : 0, e = b > skip ? b - skip : 0;
        w.first = f > see.tiles0 ? f : see.tiles0;
        const uint32_t last = e < j1 ? e : j1;
        w.count = last > w.first ? last - w.first : 0;
        return w;
    };
    const Whole block_sees = whole_for(block_lo, (int32_t)see.end - 1), wave_sees = whole_for(wave_lo, wave_hi);
    // ... widened into its buffer
    const auto put = [&](int kv, const Run& x, uint32_t buf) __attribute__((always_inline)) {
        if (!x.any) return;
        const uint32_t first = kRun * (wave % 2);
        uint8_t* to = sh.kv[kv][buf];
        if constexpr (FMT == kPageFp4) {
            const uint32_t r = first + lane / 4, s = raw_step[kv] << 23;
            if (kv && raw_step[kv] == 255) sh.odd[x.tile & 7] = x.tile + 1;
#pragma unroll
            for (int u = 0; u < D / 32; ++u) {
                const uint32_t y = raw[kv][0][u], chunk = lane % 4 * (D / 32) + u;
                *reinterpret_cast<u32x4*>(to + (kv ? place_v<D>(r, chunk) : place_k<D>(r, chunk))) =
                    u32x4{widen_fp4<0>(y, s), widen_fp4<1>(y, s), widen_fp4<2>(y, s), widen_fp4<3>(y, s)};
            }
        } else if constexpr (HALF) {
#pragma unroll
            for (int u = 0; u < NR; ++u) {
                const uint32_t r = first + (u * 1024 + lane * 16) / D, chunk = lane * 16 % D / 8;
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
            if (kv == 0) {
                if (lane < kRun) {
                    sh.steps[0][x.tile & 7][first + lane] = __uint_as_float(raw_step[0]);
                    sh.steps[1][x.tile & 7][first + lane] = __uint_as_float(raw_step[1]);
                }
                const bool nan = raw_step[1] > 0x7F800000u;
                if (nan) sh.odd[x.tile & 7] = x.tile + 1;
                const float big = __uint_as_float(max_lanes<16>(nan ? 0 : raw_step[1]));
                if (lane == 0) sh.big[x.tile & 7][wave % 2] = big;
            }
        } else if (kv && !block_sees(x.tile)) {
            // (its loads have arrived) values that are not finite are looked for where some row does not see them
            uint32_t bad = 0;
#pragma unroll
            for (uint32_t u = 0; u < kRun * CODE / 1024; ++u) {
                const u32x4 y = *reinterpret_cast<const u32x4*>(to + first * CODE + u * 1024 + lane * 16);
#pragma unroll
                for (int j = 0; j < 4; ++j) bad |= ((y[j] & 0x7F80u) == 0x7F80u) | ((y[j] & 0x7F800000u) == 0x7F800000u);
            }
            if (bad) sh.odd[x.tile & 7] = x.tile + 1;
        }
    };
    const auto arrive = [&]() {
        // LDS that other waves' loads fill is whole once each has waited for its own
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    };

    // the first keys and values are on their way before the queries are waited for: tile j0 in the place of two, its second
    const Run first = run_of(j0 - 1);
    const uint32_t second = wave / 2;  // the wave's run is of the second of two tiles
    ask(0, first, 0);
    ask(1, first, 0);
    if (thread < 8) sh.odd[thread] = 0;
    // the first turn adds the values of a tile before the first, with weights of 0
    for (uint32_t at = thread * 16; at < Tiles<FMT, D>::kBytes; at += kWaves * kWave * 16)
        *reinterpret_cast<u32x4*>(sh.kv[1][3] + at) = u32x4{0, 0, 0, 0};

    // ---- queries
    u32x4 qf[KS];
    float f = fabsf(p.scale_log2);
    {
        const uint16_t* qp = p.q.data + (uint64_t)(sq.first + tok) * p.q.ts + (uint64_t)qh * p.q.hs + 8 * hi;
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
            f = __builtin_amdgcn_ldexpf(f, -e);
        } else {
            const uint32_t turn = p.scale_log2 < 0.0f ? 0x80008000u : 0;
#pragma unroll
            for (int s = 0; s < KS; ++s) qf[s] ^= turn;
        }
        f = fmaxf(f, 1e-45f);  // of a scale of 0: all logits alike, and -inf stays what it is
    }

    // ---- running state
    f32x16 o[CB], s0, s1;
#pragma unroll
    for (int n = 0; n < CB; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[n][i] = 0.0f;
    float m = kNegInf, mu = 0.0f, l = 0.0f, top = kNegInf;
    int E = -100;  // exponent taken out of the weights (HALF), which no step so far has reached
    float wmul = __builtin_amdgcn_ldexpf(1.0f, kWeightExp + 100);
    typedef u32x4 Weights[2];  // of a tile: 16 tokens each
    Weights w0, w1;
#pragma unroll
    for (int k = 0; k < 2; ++k) w0[k] = w1[k] = 0;

    // whether the row sees token t0 + 4 hi + c
    struct Sight {
        int32_t past, left, sunk_to;
        __device__ __forceinline__ bool operator()(int32_t c) const { return (c <= past) & ((c > left) | (c < sunk_to)); }
    };
    const auto sight_of = [&](uint32_t t0) {
        Sight x;
        x.past = pos - (int32_t)t0 - 4 * (int32_t)hi;
        x.left = p.window ? x.past - (int32_t)p.window : -0x7FFFFFFF;
        x.sunk_to = p.window ? (int32_t)p.sinks - (int32_t)t0 - 4 * (int32_t)hi : 0;
        return x;
    };
    // keys of a product step: 32 tokens, 16 channels
    const auto keys = [&](uint32_t buf, int k) {
        return *reinterpret_cast<const u32x4*>(sh.kv[0][buf] + place_k<D>(col, 2 * k + hi));
    };
    // values of a product: 32 channels (block n), 16 tokens. A read gives four tokens of one channel to a lane: token
    // 4 hi + (lane % 16) / 4 of each 8, channels of 64 bytes
    const uint32_t i16 = lane & 15;
    const auto values = [&](uint32_t buf, int k, int n) {
        const uint32_t chunk = 4 * n + (lane >> 4 & 1) * 2 + (i16 & 3) / 2;
        const uint32_t t = 16 * k + 4 * hi + i16 / 4;
        const auto part = [&](uint32_t token) {
            return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                 (KVC_LDS s16x4*)(sh.kv[1][buf] + place_v<D>(token, chunk) + (i16 & 1) * 8)));
        };
        const u32x2 a = part(t), c = part(t + 8);
        return u32x4{a.x, a.y, c.x, c.y};
    };
    // a tile's logits from its products: their keys' steps, and the mask (behind the last tile, of all of them, whatever the
    // buffer holds)
    const auto logits = [&](uint32_t j, f32x16& x) __attribute__((always_inline)) {
        if constexpr (HALF) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const f32x4 ks = *reinterpret_cast<const f32x4*>(&sh.steps[0][j & 7][8 * w + 4 * hi]);
#pragma unroll
                for (int c = 0; c < 4; ++c) x[4 * w + c] *= ks[c];
            }
        }
        if (!wave_sees(j)) {
            Sight sees = sight_of(start_of(j));
            if (j >= j1) sees.past = -1;
#pragma unroll
            for (int c = 0; c < 16; ++c) x[c] = sees(8 * (c / 4) + c % 4) ? x[c] : kNegInf;
        }
    };
    // Values of a buffer (8 bits: their steps) that are not finite, in a tile that some row sees only part of: a row that
    // sees one is NaN in its channel, which is noted here (bit 16 n + 4 j + c of the lane's channels), and it becomes 0.
    // (Every wave comes by.)
    uint64_t lost = 0;
    const auto take_out = [&](uint32_t j) __attribute__((always_inline)) {
        const uint32_t buf = (j - j0) & 3;
        uint8_t* vt = sh.kv[1][buf];
        const Sight sees = sight_of(start_of(j));
#pragma unroll 1
        for (int t = 0; t < (int)kTokens; ++t) {
            if (!sees(t - 4 * (int32_t)hi)) continue;
            if constexpr (HALF) {
                if (__builtin_isnan(sh.steps[HALF][j & 7][t])) lost = ~0ull;
            } else {
#pragma unroll 1
                for (int i = 0; i < 4 * CB; ++i) {
                    const u32x2 y = *reinterpret_cast<const u32x2*>(vt + place_v<D>(t, i) + 8 * hi);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if ((y[c / 2] >> (16 * (c % 2)) & 0x7F80u) == 0x7F80u) lost |= 1ull << (4 * i + c);
                }
            }
        }
        __syncthreads();
        if constexpr (HALF) {
            if (thread < kTokens) {
                float& x = sh.steps[1][j & 7][thread];
                x = __builtin_isnan(x) ? 0.0f : x;
            }
        } else {
            for (uint32_t at = thread * 16; at < Tiles<FMT, D>::kBytes; at += kWaves * kWave * 16) {
                u32x4 y = *reinterpret_cast<u32x4*>(vt + at);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    y[c] = (y[c] & 0x7F80u) == 0x7F80u ? y[c] & 0xFFFF0000u : y[c];
                    y[c] = (y[c] & 0x7F800000u) == 0x7F800000u ? y[c] & 0xFFFFu : y[c];
                }
                *reinterpret_cast<u32x4*>(vt + at) = y;
            }
        }
        __syncthreads();
    };
    // adds a tile's weighted values
    const auto add_values = [&](uint32_t buf, const Weights& w) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int n = 0; n < CB; ++n) o[n] = mfma<FMT>(values(buf, k, n), w[k], o[n]);
    };

    // ---- One tile's part of the pipeline: the products of the next tile's keys (into `next`), this one's weights (from
    // `now`, into `w`) and the values of the one before (weighted by `before`) are independent, and go side by side: two
    // products beside two weights (four with 64 channels), first those of keys, so that the next tile's largest logit is
    // found beside those of values. What two products read from LDS was asked for two products before (`op`: that of the
    // first two). (The barriers keep the compiler from asking for everything at once, which spills 100 registers.)
    const auto first_keys = [&](uint32_t buf, u32x4 (&op)[4]) __attribute__((always_inline)) {
        op[0] = keys(buf, 0);
        op[1] = keys(buf, 1);
    };
    const auto turn = [&](uint32_t j, auto keys_in, auto values_in, f32x16& now, f32x16& next, Weights& before, Weights& w,
                          u32x4 (&op)[4]) __attribute__((always_inline)) {
        constexpr uint32_t kb = decltype(keys_in)::value, vb = decltype(values_in)::value;
        constexpr int PAIRS = 8 / KS;  // of weights beside two products
        const uint32_t sb = j & 7;
        u32x2 vs[2][HALF ? PAIRS : 1];
        const auto steps_of = [&](int k, u32x2 (&x)[HALF ? PAIRS : 1]) {
            if constexpr (HALF) {
#pragma unroll
                for (int c = 0; c < PAIRS; ++c) {
                    const int v = PAIRS * k + c;  // tokens of elements 2 v, 2 v + 1 of 16
                    x[c] = *reinterpret_cast<const u32x2*>(&sh.steps[1][sb][8 * (v / 2) + 4 * hi + 2 * (v % 2)]);
                }
            }
        };
        // (steps count for their tile's weights, values when they are added)
        const uint32_t odd = HALF ? j : j - 1;
        if (__builtin_expect(!block_sees(odd), 0)) {
            if (j >= j0 + !HALF && j < j1 + !HALF && sh.odd[odd & 7] == odd + 1) take_out(odd);
        }
        bool move = top > m + kSlack;
        // steps of the values are brought into binary16's range by 2^-E; those that the row sees count for E
        float big = 0.0f;
        if constexpr (HALF) {
            if (wave_sees(j)) {
                const float2 y = *reinterpret_cast<const float2*>(sh.big[j & 7]);
                big = fmaxf(y.x, y.y);
            } else if (j < j1) {
                const Sight sees = sight_of(start_of(j));
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const f32x4 y = *reinterpret_cast<const f32x4*>(&sh.steps[1][j & 7][8 * v + 4 * hi]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) big = fmaxf(big, sees(8 * v + c) ? y[c] : 0.0f);
                }
            }
            move |= big >= __builtin_amdgcn_ldexpf(1.0f, E);
        }
        if (__ballot(move) != 0) {
            // (the weights before are relative to m as it was)
            add_values(vb, before);
#pragma unroll
            for (int k = 0; k < 2; ++k) before[k] = 0;
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
#pragma unroll
        for (int i = 0; i < 16; ++i) next[i] = 0.0f;
        steps_of(0, vs[0]);
        float largest = kNegInf;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int q = 2 * k + 2 + x;  // of KS products of keys, then KS of values
                if (q < KS)
                    op[q % 4] = keys(kb, q);
                else if (q < 2 * KS)
                    op[q % 4] = values(vb, (q - KS) / CB, (q - KS) % CB);
            }
            if (k + 1 < KS) steps_of(k + 1, vs[(k + 1) & 1]);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int q = 2 * k + x, v = q - KS;
                if (q < KS)
                    next = mfma<FMT>(op[q % 4], qf[q % KS], next);
                else
                    o[v % CB] = mfma<FMT>(op[q % 4], before[v / CB & 1], o[v % CB]);
            }
#pragma unroll
            for (int x = 0; x < PAIRS; ++x) {
                const int v = PAIRS * k + x;
                float e[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    e[c] = __builtin_amdgcn_exp2f(fmaf(now[2 * v + c], f, -mu));
                    l += e[c];
                    if constexpr (HALF) e[c] = e[c] * __uint_as_float(vs[k & 1][x][c]) * wmul;
                }
                w[v / 4][v % 4] = HALF ? pack_half2(e[0], e[1]) : pack_bf16x2(e[0], e[1]);
            }
            // added up and packed here, not at the end, where all weights would have to be kept
            asm volatile("" : "+v"(l));
#pragma unroll
            for (int x = 0; x < PAIRS; ++x) asm volatile("" : "+v"(w[(PAIRS * k + x) / 4][(PAIRS * k + x) % 4]));
            constexpr int LEFT = KS / 2 - 1;  // steps behind the first with values: the next logits are there
            if (k > KS / 2) {
#pragma unroll
                for (int c = 16 * (k - KS / 2 - 1) / LEFT; c < 16 * (k - KS / 2) / LEFT; ++c) largest = fmaxf(largest, next[c]);
                asm volatile("" : "+v"(largest));
            }
            __builtin_amdgcn_sched_barrier(0);
            if (k == KS / 2) logits(j + 1, next);
        }
        top = largest * f;
    };

    // ---- Two tiles, j and j + 1, between barriers: keys j + 1, j + 2 and values j - 1, j are there, keys j + 3, j + 4 and
    // values j + 1, j + 2 on their way
    if (j0 < j1) {
        Run ahead = run_of(j0 + 1);
        __syncthreads();  // `odd` is cleared, by one wave for all
        if (FMT != kPageBf16) {  // (their registers are needed again)
            put(0, first, 0);
            put(1, first, 0);
        }
        ask(0, ahead, 1 + second);
        arrive();
        if (FMT == kPageBf16) put(1, first, 0);
        put(0, ahead, 1 + second);
        Run then = run_of(j0 + 3);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 16; ++i) s0[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < KS; ++k) s0 = mfma<FMT>(keys(0, k), qf[k], s0);
        logits(j0, s0);
        top = kNegInf;
#pragma unroll
        for (int c = 0; c < 16; ++c) top = fmaxf(top, s0[c]);
        top *= f;
        u32x4 op[4];
        // four tiles a turn of the loop, so that their buffers are known when this is compiled
        const auto two = [&](uint32_t j, auto first_buffer) __attribute__((always_inline)) {
            constexpr uint32_t B = decltype(first_buffer)::value;
            first_keys((B + 1) & 3, op);
            ask(1, ahead, (B + 1 + second) & 3);
            ask(0, then, (B + 3 + second) & 3);
            const Run behind = ahead;
            ahead = then;
            then = run_of(j + 5);
            turn(j, std::integral_constant<uint32_t, (B + 1) & 3>{}, std::integral_constant<uint32_t, (B + 3) & 3>{}, s0, s1, w1, w0, op);
            first_keys((B + 2) & 3, op);
            turn(j + 1, std::integral_constant<uint32_t, (B + 2) & 3>{}, std::integral_constant<uint32_t, B>{}, s1, s0, w0, w1, op);
            arrive();
            put(1, behind, (B + 1 + second) & 3);
            put(0, ahead, (B + 3 + second) & 3);
            __syncthreads();
        };
        for (uint32_t j = j0;;) {
            two(j, std::integral_constant<uint32_t, 0>{});
            j += 2;
            if (j >= j1) break;
            two(j, std::integral_constant<uint32_t, 2>{});
            j += 2;
            if (j >= j1) break;
        }
        if ((j1 - j0) % 2 == 0) {  // (else the last tile's values went beside a tile that is none)
            if (!HALF && !block_sees(j1 - 1) && sh.odd[(j1 - 1) & 7] == j1) take_out(j1 - 1);
            add_values((j1 - 1 - j0) & 3, w1);
        }
    }

    // ---- output
    if (__ballot(lost != 0) != 0) {
#pragma unroll
        for (int n = 0; n < CB; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[n][i] = lost >> (16 * n + i) & 1 ? __builtin_nanf("") : o[n][i];
    }
    l = over_pair(l, [](float a, float c) { return a + c; });
    if (HALF) {
        const float down = __builtin_amdgcn_ldexpf(1.0f, E - kWeightExp);
#pragma unroll
        for (int n = 0; n < CB; ++n) o[n] *= down;
    }
    if (cut) {
        // a share's first piece continues a block, or its last begins one
        if (has_row) {
            float* to = p.part + ((uint64_t)(2 * share + (part0 == 0)) * p.H + h) * (kRows * (D + 2));
#pragma unroll
            for (int n = 0; n < CB; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<f32x4*>(to + ((n * kWaves + wave) * 4 + j) * (4 * kWave) + 4 * lane) =
                        f32x4{o[n][4 * j], o[n][4 * j + 1], o[n][4 * j + 2], o[n][4 * j + 3]};
            if (hi == 0) *reinterpret_cast<float2*>(to + kRows * D + 2 * my_row) = make_float2(m, l);
        }
        continue;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    if (p.lse && has_row && hi == 0) p.lse[(uint64_t)(sq.first + tok) * p.Hq + qh] = (m + log2f(l)) * 0.69314718055994531f;
    // rows go through LDS, so that they are written in one piece
    constexpr uint32_t LINE = 2 * D + 16, LPR = 2 * D / 16;  // bytes of a row there; lanes that write one
    static_assert(kRows * LINE <= sizeof(sh.kv));
    uint8_t* mine = &sh.kv[0][0][0] + wave * 32 * LINE;
    __syncthreads();
#pragma unroll
    for (int n = 0; n < CB; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<u32x2*>(mine + col * LINE + 2 * (32 * n + 8 * j + 4 * hi)) =
                u32x2{pack_bf16x2(o[n][4 * j] * inv, o[n][4 * j + 1] * inv), pack_bf16x2(o[n][4 * j + 2] * inv, o[n][4 * j + 3] * inv)};
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (uint32_t u = 0; u < 32 * LPR / kWave; ++u) {
        const uint32_t r = u * (kWave / LPR) + lane / LPR, piece = lane % LPR, at = wave * 32 + r;
        const uint32_t to_tok = (row0 + at) / p.group, to_head = h * p.group + (row0 + at) % p.group;
        if (at < nrows)
            *reinterpret_cast<u32x4*>(p.out.data + (uint64_t)(sq.first + to_tok) * p.out.ts + (uint64_t)to_head * p.out.hs + 8 * piece) =
                *reinterpret_cast<const u32x4*>(mine + r * LINE + 16 * piece);
    }
    if constexpr (!SHARED) return;
    }
}

// Joins what shares have of a block that is cut up: a workgroup 32 channels, whose lanes hold what those of the shares held.
template <int D>
__global__ __launch_bounds__(kBlockThreads) void prompt_join_kernel(PromptParams p) {
    fetch_arguments<sizeof(PromptParams)>();
    constexpr uint32_t CB = D / 32;
    const uint32_t h = blockIdx.x % p.H, n = blockIdx.x / p.H % CB, place = blockIdx.x / p.H / CB;
    const u32x2 info = *(const __attribute__((address_space(4))) u32x2*)(uint64_t)(p.info + (uint64_t)place * p.H + h);
    const uint32_t b = sequence_of(p, place);
    if (b >= p.n) return;
    const Sequence sq = uniform(sequence_at<false>(p, p.n - 1 - b), 0);
    const uint32_t block = place - first_block(p, b, sq.first);
    if (block >= sq.blocks || info.y == 0) return;  // none, or written already
    if (info.x >= p.shares || info.y > p.shares - info.x) return;  // (starts were wrong: no share wrote it)
    const uint32_t lane = lane_id(), wave = threadIdx.x / kWave, hi = lane >> 5, r = wave * 32 + lane % 32;
    const uint32_t row = block * kRows + r, parts = info.y;
    if (row >= sq.m * p.group) return;  // (with its neighbour, which holds the row's other channels)
    // part 0 is the last piece of its share, the others the first of theirs
    const auto part_of = [&](uint32_t i) {
        return p.part + ((uint64_t)(i ? 2 * (info.x + i) : 2 * info.x + 1) * p.H + h) * (kRows * (D + 2));
    };
    float M = kNegInf;
#pragma unroll 4
    for (uint32_t i = 0; i < parts; ++i) M = fmaxf(M, part_of(i)[kRows * D + 2 * r]);
    const float Mu = M == kNegInf ? 0.0f : M;
    float total = 0.0f;
    f32x4 y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = 0.0f;
#pragma unroll 2
    for (uint32_t i = 0; i < parts; ++i) {
        const float* from = part_of(i);
        const float2 ml = *reinterpret_cast<const float2*>(from + kRows * D + 2 * r);
        const float w = __builtin_amdgcn_exp2f(ml.x - Mu);
        total = fmaf(ml.y, w, total);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f32x4 v = *reinterpret_cast<const f32x4*>(from + ((n * kWaves + wave) * 4 + j) * (4 * kWave) + 4 * lane);
            if (ml.x == kNegInf) v = 0.0f;  // (a part without tiles has no sums)
            y[j] += v * w;
        }
    }
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    const uint32_t tok = sq.first + row / p.group, qh = h * p.group + row % p.group;
    uint16_t* to = p.out.data + (uint64_t)tok * p.out.ts + (uint64_t)qh * p.out.hs + 32 * n;
    // two lanes hold channels 8 j + 4 hi to + 3: one takes all of j, the other of j + 1
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
        u32x4 z;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const auto q = __builtin_amdgcn_permlane32_swap(pack_bf16x2(y[j][2 * c] * inv, y[j][2 * c + 1] * inv),
                                                            pack_bf16x2(y[j + 1][2 * c] * inv, y[j + 1][2 * c + 1] * inv), false, false);
            z[c] = q[0];
            z[2 + c] = q[1];
        }
        *reinterpret_cast<u32x4*>(to + 8 * (j + hi)) = z;
    }
    if (p.lse && n == 0 && hi == 0) p.lse[(uint64_t)tok * p.Hq + qh] = (M + log2f(total)) * 0.69314718055994531f;
}

template <int D, bool SHARED>
hipError_t launch_of(uint32_t format, const PromptParams& p, uint32_t grid, hipStream_t stream) {
    const auto f = format == kPageBf16   ? prompt_kernel<kPageBf16, D, SHARED>
                   : format == kPageInt8 ? prompt_kernel<kPageInt8, D, SHARED>
                   : format == kPageFp8  ? prompt_kernel<kPageFp8, D, SHARED>
                                         : prompt_kernel<kPageFp4, D, SHARED>;
    return launch_kernel(f, dim3(grid), dim3(kWaves * kWave), stream, p);
}

// Workgroups of 4 waves that the GPU holds at once. Tiles are shared out up to 5/4 as many blocks: more balance one another,
// and beginning a piece of a block costs what eight tiles cost. Blocks shared out and not, us: 504 blocks of 512 places (one
// prompt of 2000 tokens, 8 kv heads of 128, 4 heads each, bf16) 64 and 80, 600 93 and 98, 752 125 and 96, 1500 361 and
// 309; where contexts differ, 712 (chunks of four prompts, int8) 215 and 244.
constexpr uint64_t places_of(uint32_t d) { return kCus * workgroups(d); }
// Few new tokens of each sequence (their rows, times the heads that share a kv head, in the mean of all): a call is then
// memory's, and the kernel for one new token takes them, 32 rows at a time. That kernel and the one here, us, 8 kv heads of
// 128: 15 sequences behind 8192 tokens, 32 rows e4m3 56 and 112, bf16 106 and 112, 64 rows 98 and 116, 160 and 115, 80 rows 134
// and 120, 239 and 118; 4 such sequences, 64 rows 29 and 63, 34 and 52, 80 rows 46 and 65, 73 and 53; one of 32 rows behind
// 4000 tokens e4m3 15 and 32, behind 400 12 and 20, and, with a second launch that joins what it shared out, behind 100 13 and
// 11. (Rows that belong to no sequence count as well: a quarter more.) So 80 is too many for bf16 where there are more
// than a few sequences (60 behind 2000, 64 rows: 207 and 98); a rule that knows the format and the sequences is not here yet.
constexpr uint64_t kFewRows = 80;
constexpr uint64_t kFewTokens = 256;

}  // namespace

PromptPlan prompt_plan(uint32_t n_seqs, uint32_t n_tokens, uint32_t H, uint32_t Hq, uint32_t d, uint64_t max_tokens,
                       uint32_t window, uint32_t sinks) {
    const uint64_t group = Hq / H;
    PromptPlan a{};
    a.blocks = n_tokens * group / kRows + n_seqs;
    a.bytes = a.room = 256;
    // with a window, a block's rows see the tokens of one row and as many more as the block has tokens
    const uint64_t seen = window ? seen_tokens(max_tokens, (uint64_t)window + kRows / group, sinks) : max_tokens;
    const bool can = seen > kMinShare * kTokens;
    const uint64_t places = places_of(d), shares = (places + H - 1) / H, few_blocks = 5 * places / 4;
    if (can && H * a.blocks < few_blocks) a.shares = (uint32_t)shares;
    // a share leaves two parts of blocks at most
    const uint64_t parts = align_up(2 * shares * H * (kRows * (d + 2) * 4), 256);
    const uint64_t info = align_up(a.blocks * H * 8, 256);
    if (a.shares) a.bytes = parts + info;
    if (can && H < few_blocks) a.room = parts + align_up((a.blocks < few_blocks / H + 1 ? a.blocks : few_blocks / H + 1) * H * 8, 256);
    const uint64_t rows = n_tokens * group, most = kFewRows * n_seqs, few = rows < most ? rows : most;
    const AttendPlan many = many_attend_plan(n_seqs, n_tokens, H, Hq, d, max_tokens, window, sinks);
    // (what its kernels count with 32 bits, wherever the sequences start, and a wave's threads of each row)
    a.few = rows <= most && max_tokens > kFewTokens && rows * H < 1ull << 24 && (uint64_t)n_seqs * (rows / 16 + 1) * (max_tokens / 128 + 1) < 1ull << 31;
    if (a.few) a.bytes = many.bytes(d);
    const uint64_t room = many_attend_room(n_seqs, few, H, d, max_tokens);
    if (room > a.room) a.room = room;
    return a;
}

hipError_t launch_attend_prompt(const PromptArgs& a, const PromptPlan& plan, hipStream_t stream) {
    if (plan.few) {
        AttendArgs b{};
        b.n = a.n;
        b.H = a.H;
        b.Hq = a.Hq;
        b.d = a.d;
        b.q = a.q;
        b.out = a.out;
        b.scale = a.scale;
        b.lse = a.lse;
        b.ws = a.ws;
        b.status = a.status;
        b.tail = a.tail;
        b.starts = a.starts;
        b.tokens = a.rows;
        return launch_attend(b, stream);
    }
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
    p.shares = plan.shares;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.part = static_cast<float*>(a.ws);
    // behind the parts
    p.info = reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.ws) + align_up(2ull * plan.shares * a.H * (kRows * (a.d + 2) * 4), 256));
    const uint32_t grid = (uint32_t)((plan.shares ? plan.shares : plan.blocks) * a.H);
    if (!plan.shares)
        return a.d == 64 ? launch_of<64, false>(lay.format, p, grid, stream) : launch_of<128, false>(lay.format, p, grid, stream);
    const hipError_t e = a.d == 64 ? launch_of<64, true>(lay.format, p, grid, stream) : launch_of<128, true>(lay.format, p, grid, stream);
    if (e != hipSuccess) return e;
    const auto join = a.d == 64 ? prompt_join_kernel<64> : prompt_join_kernel<128>;
    return launch_kernel(join, dim3((uint32_t)(plan.blocks * a.H * (a.d / 32))), dim3(kBlockThreads), stream, p);
}

}  // namespace kvc
