// tree_attention.hpp -- attention of drafted tokens over a paged cache.
//
// For row n (a node and a query head) over the tokens t it sees:
//     s = scale q.k_t,  out = sum_t 2^(s' - M) v_t / sum_t 2^(s' - M),
// s' = s log2(e), with the running maximum M and sum of an online softmax in
// float32. All query heads of a kv head and all nodes are rows of one product,
// so a tile of keys and values is read once for all of them.
//
// Products use the 32x32x16 matrix instruction (16x16x32 where a wave has 16
// rows, with half the registers and exponentials), transposed: S^T = K Q^T puts one
// row n in each lane column (lane % 32), 16 of 32 tokens in a lane and the
// other 16 in lane ^ 32, so maxima and sums are lane-local but for one
// exchange. The exponentials are then already the operand of O^T = V^T P^T: a
// product does not mind the order of the tokens it sums over, so V^T is read
// in the order that S^T left them in, with the transposing LDS load.
//
// A team of waves walks its tokens in tiles: while one tile is computed, the
// next is on its way from memory into registers (rows looked up through the
// page table a tile earlier), and is converted to 16 bits on its way into the
// LDS, once for all its waves. With few rows a team is one wave and needs no
// barrier; the block's waves take tiles in turn and join at the end. 8-bit
// elements stay whole: the scale of a key multiplies its scores, and the scale
// of a value joins the exponent,
//     w_t = 2^(s'_t + log2 c_t - M),  out = sum_t w_t code_t / sum_t w_t / c_t,
// so that w is at most 1 (2^8 until M follows) whatever the scales are. Where
// scales are so far apart that some w vanish whose w / c do not, the piece is
// gone through again without them for the sum, and once more for the output.
// (Sums that bear any scales in one pass, of squared roots of w / c, cost all
// others: 32 sequences x 32 rows 130.7 us / 123.5.) P is rounded to the type
// of V in the product (float16 for 8-bit caches, which hold those exactly):
// relative 2^-11 or 2^-8 a term, the step of the output's own type.
//
// The tiles of all sequences, heads and blocks of rows are shared out evenly
// over as many blocks as the card holds at once, whatever the lengths: a block
// takes a run of tiles, which may end one segment and begin the next, and
// writes the sums of every piece; combine_kernel joins a segment's pieces in
// order. (With a fixed grid of chunks instead, 32 sequences of 1500 to 16384
// tokens kept the compute units half busy: 231 us.)
//
// What it takes, without the joining:
//   32 sequences of 1500 to 16384 tokens, 8 kv heads x 32 rows of 128, int8:
//     608 MB in 117.6 us (5.2 TB/s). Two waves a SIMD, each with its chain of
//     loads, conversion, products and exponentials: vector instructions fill
//     40 % of the cycles, the LDS is busy for 27 %, the matrix unit for 13 %;
//     memory alone would need 84 us. More waves do not fit the registers.
//   4 sequences of 8192 tokens, 8 kv heads x 512 rows of 128, bf16:
//     64 GFLOP in 100 us (640 TFLOP/s, half of a large product's rate):
//     the matrix unit is busy for 27 % of the cycles, vector instructions
//     fill 26 %, the LDS 22 %; exponentials wait for products, products for
//     exponentials, and the waves for each other's tiles.
//   1 sequence of 8191 tokens, 8 kv heads x 4 rows of 128, float16: 34 MB in
//     12 us: latency, of the plan, the page, the rows and the joined sums.
//   Up to 16 rows a kv head of 128: 32 sequences of 1500 to 16384 tokens, 4 rows,
//     bf16 1173 MB in 194 us (6.1 TB/s), int8 605 MB in 104.5 us (5.8 TB/s).
//   Heads of 256, 8 sequences of 3000 to 8000 tokens, bf16: 4 rows 361 MB in
//     68 us (5.3 TB/s), 64 rows 183 MB in 53.7 us (3.4 TB/s, 215 TFLOP/s).
#pragma once

#include "decode_common.hpp"
#include "launch.hpp"

namespace libred {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <class T>
struct Mma;
template <>
struct Mma<F16> {
    static __device__ __forceinline__ f32x16 dot(u32x4 a, u32x4 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
    }
    static __device__ __forceinline__ f32x4 dot(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
    }
    static constexpr uint32_t kExponent = 0x7C00u;
};
template <>
struct Mma<BF16> {
    static __device__ __forceinline__ f32x16 dot(u32x4 a, u32x4 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    }
    static __device__ __forceinline__ f32x4 dot(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
    }
    static constexpr uint32_t kExponent = 0x7F80u;
};

// The elements of a cache: how many bytes, and 4 of them as 16-bit values.
struct Cached16 {
    static constexpr int kBytes = 2;
};
struct CachedI8 {
    static constexpr int kBytes = 1;
    template <class T>
    static __device__ __forceinline__ u32x2 widen4(uint32_t w) {
        if constexpr (std::is_same_v<T, F16>) {
            // The biased byte as the low bits of 1024 + b, less 1152.
            const uint32_t b = w ^ 0x80808080u;
            const f16x2 c = {(_Float16)1152.f, (_Float16)1152.f};
            return u32x2{__builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, b, 0x04010400u)) - c),
                         __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, b, 0x04030402u)) - c)};
        } else {
            return u32x2{Mma<BF16>::pack((float)(int8_t)w, (float)(int8_t)(w >> 8)),
                         Mma<BF16>::pack((float)(int8_t)(w >> 16), (float)(int8_t)(w >> 24))};
        }
    }
};
struct CachedE4M3 {
    static constexpr int kBytes = 1;
    template <class T>
    static __device__ __forceinline__ u32x2 widen4(uint32_t w) {
        if constexpr (std::is_same_v<T, F16>)
            return u32x2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, false)),
                         __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, true))};
        else
            return u32x2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, false)),
                         __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, true))};
    }
};

// Combine the values of the lanes that share a row: lane ^ 32, and lane ^ 16
// where a row of the tile is spread over four. Every lane gets the result.
template <int PARTS, class F>
__device__ __forceinline__ float join_parts(float v, F op) {
    const unsigned a = __builtin_bit_cast(unsigned, v);
    const auto s = __builtin_amdgcn_permlane32_swap(a, a, false, false);
    // Elements of a vector go through variables: a bit cast of s[1] itself
    // reads element 0.
    const unsigned s0 = s[0], s1 = s[1];
    v = op(__builtin_bit_cast(float, s0), __builtin_bit_cast(float, s1));
    if constexpr (PARTS == 4) {
        const unsigned c = __builtin_bit_cast(unsigned, v);
        const auto q = __builtin_amdgcn_permlane16_swap(c, c, false, false);
        const unsigned q0 = q[0], q1 = q[1];
        v = op(__builtin_bit_cast(float, q0), __builtin_bit_cast(float, q1));
    }
    return v;
}

// A value that is the same in all lanes, as one the compiler knows to be.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The kernel's arguments, as memory that the compiler has not seen yet: what is
// needed at the two ends of a segment is loaded there and holds no registers in
// between.
typedef const __attribute__((address_space(4))) TreeAttention* Arguments;
__device__ __forceinline__ Arguments arguments_again() {
    auto p = __builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return (Arguments)p;
}

constexpr float kLazy = 8.f;  // how far (in powers of 2) scores may pass M before M follows
// Scales of values between these, and a row of zeros taken as kZeroScale (it
// should not raise M), are never so far apart that a weight vanishes (exp2
// gives 0 below 2^-126) whose share of the sum, w / c, is above 2^-56.
constexpr float kLeastScale = 0x1p-50f, kMostScale = 0x1p10f, kZeroScale = 0x1p-60f;

// RW rows a wave (the side of its matrix instruction), WM waves of different
// rows, WT of different tokens, TS tokens a tile.
template <class C, int DP, int RW, int WM, int WT, int TS>
struct AttentionTile {
    static constexpr int kThreads = kWave * WM * WT;
    static constexpr int kTokens = WT * TS;
    static constexpr int kRows = RW * WM;
    static constexpr int kPerLoad = 16 / C::kBytes;  // elements of a 16-byte load
    static constexpr int kRowLoads = DP / kPerLoad;
    // Place p * kRowLoads + j of a row in the LDS holds the 8 elements that are
    // part p of load j: the two parts of a load of 8-bit elements, 32 bytes
    // once widened, are stored apart so that 8 lanes store 128 bytes in a row.
    // (Side by side they met in the banks, a third of the LDS's cycles: 16
    // sequences of 2000 to 8000 tokens, 8 kv heads x 4 rows of 128, e4m3, 40.1
    // us / 37.9.) The order of k's elements is q's too; dim_of() undoes v's.
    static constexpr int dim_of(int c) {
        return kPerLoad == 8 ? c : c / 8 % kRowLoads * kPerLoad + c / 8 / kRowLoads * 8 + c % 8;
    }
    // A team of waves shares a tile of TS tokens: the waves_m waves of
    // different rows, or one wave, which then needs no barriers.
    static constexpr int kTeam = kWave * WM;
    static constexpr int kLoads = (TS * kRowLoads + kTeam - 1) / kTeam;
    // Tiles a team holds in the LDS: with barriers two, so that one is written
    // while the other is read and there is one barrier a tile.
    static constexpr int kHeld = WM > 1 ? 2 : 1;
    // Row pitches in the LDS (bytes): 16 times an odd number, so that 16-byte
    // reads down a column of 8 rows meet all banks; 64 more than a multiple
    // of 128, so that the transposing reads of 4 rows times 64 bytes do.
    static constexpr int kPitchK = DP * 2 + 16;
    static constexpr int kPitchV = (DP * 2) % 128 == 64 ? DP * 2 : DP * 2 + 64;
    static constexpr int kTileBytes = TS * (kPitchK + kPitchV);
    static constexpr int kPitchO = DP + 4;  // floats
    static constexpr int kOutBytes = WT > 1 ? WM * WT * RW * kPitchO * 4 : 0;
    static constexpr int kAllTiles = WT * kHeld * kTileBytes;
    static constexpr int kBytes = kAllTiles > kOutBytes ? kAllTiles : kOutBytes;
};

template <class T, class C, int DP, int RW, int WM, int WT, int TS>
__global__ __launch_bounds__(kWave* WM* WT, DP <= 128 || (RW == 16 && WM > 1) ? 2 : 1) void tree_attention_kernel(TreeAttention a) {
    using S = AttentionTile<C, DP, RW, WM, WT, TS>;
    constexpr bool kScaled = C::kBytes == 1;
    using VT = std::conditional_t<kScaled, F16, T>;
    // A row lies in PARTS lanes (RW apart), which hold X of 32 tokens each, in
    // fours: value x is of token 4 PARTS (x / 4) + 4 part + x % 4. One product
    // takes KD elements of q and k, and XP = 8 values a lane of P.
    constexpr int PARTS = kWave / RW, X = 32 / PARTS, KD = 8 * PARTS;
    constexpr int TT = S::kTokens, KS = DP / KD, DT = DP / RW, SUB = TS / 32, OX = RW * RW / kWave;
    using Acc = std::conditional_t<RW == 32, f32x16, f32x4>;
    static_assert(WM == 1 || WT == 1, "a team is a wave or the block");
    constexpr int HELD = S::kHeld, NL = S::kLoads;
    __shared__ __align__(16) char tile[S::kBytes];
    __shared__ uint32_t offs_all[WT][4][TS];  // where the rows of a tile's tokens start, in 16 bytes
    __shared__ uint64_t held[WT][4];           // which of them are in the cache
    __shared__ __align__(16) float factors[WT][HELD][3][kScaled ? TS : 4];  // of keys; of values: logarithm, inverse
    __shared__ float red[2][WM * WT][RW];
    // Infinities or NaN among a node's values, or for its scale (kOdd), which some
    // rows may not see; for the scale of a token that all rows see (kLost);
    // scales beyond kLeastScale and kMostScale (kBeyond).
    constexpr int kOdd = 1, kLost = 2, kBeyond = 4;
    __shared__ int notes;
    __shared__ float unscaled[2][kScaled ? S::kRows : 1];  // maxima and sums of pass 1

    // One argument of every 64-byte line, so that all lines are asked for at
    // once: fetched one after the other as they are met, the arguments alone
    // take several microseconds of a small call.
    asm volatile("" ::"s"(a.q), "s"(a.q_head), "s"(a.cache.k), "s"(a.cache.scale_head_stride), "s"(a.lens), "s"(a.blocks), "s"(a.plan));
    const int tid = threadIdx.x, wave = uniform(tid / kWave), lane = tid % kWave, n = lane % RW, part = lane / RW;
    const int wm = wave % WM, wt = wave / WM;
    const int tm = WM == 1 ? lane : tid;  // in the team
    char* const tiles_lds = tile + wt * HELD * S::kTileBytes;
    auto& offs = offs_all[wt];
    const int D = a.cache.dim, group = a.group, M = a.nodes * group, heads = a.cache.heads;
    const bool direct = a.blocks == 0;
    const int per_seq = heads * a.row_blocks;  // segments of a sequence

    // This block's share of the tiles: [now, end) of all segments' tiles
    // (below 2^31, which the entry point checks).
    int b = 0, seg = 0, skip = 0;  // sequence, segment in it, tiles of that segment that are another's
    int now = 0, end = 1;
    int len, count;  // of sequence b
    // Blocks are dealt to the XCDs in turn; each XCD takes a run of shares, so
    // that the blocks of rows of one head read its tokens through one L2.
    const int share = direct || gridDim.x % kXcds ? blockIdx.x : blockIdx.x % kXcds * (gridDim.x / kXcds) + blockIdx.x / kXcds;
    auto load_sequence = [&](int q, int* q_len, int* q_count) {
        const int c = a.count ? min(max(a.count[q], 0), a.nodes) : a.nodes;
        *q_len = max(a.lens[q], 0);
        *q_count = c;
    };
    auto tokens_of = [&](int q_len, int q_count) { return (int)min((int64_t)q_len + q_count, (int64_t)a.max_tokens); };
    if (direct) {
        b = blockIdx.x / per_seq, seg = blockIdx.x % per_seq;
        load_sequence(b, &len, &count);
    } else {
        // 64 sequences at a time, one a lane; `upto` is the running sum of
        // their tiles.
        int at_len = 0, at_count = 0, own = 0, upto = 0;
        auto group_of = [&](int q) {
            at_len = at_count = own = 0;
            if (q + lane < a.batch) {
                load_sequence(q + lane, &at_len, &at_count);
                own = at_count > 0 ? (tokens_of(at_len, at_count) + TT - 1) / TT : 0;
            }
            upto = own;
            upto += dpp_move<0x111, 0xF>(0, upto);  // shifted by 1, 2, 4 and 8 in rows of 16
            upto += dpp_move<0x112, 0xF>(0, upto);
            upto += dpp_move<0x114, 0xF>(0, upto);
            upto += dpp_move<0x118, 0xF>(0, upto);
            upto += dpp_move<0x142, 0xA>(0, upto);  // rows 0 and 2 into 1 and 3
            upto += dpp_move<0x143, 0xC>(0, upto);  // the first half into the second
        };
        int all = 0;
        for (int q = 0; q < a.batch; q += kWave) {
            group_of(q);
            all += read_lane(upto, kWave - 1);
        }
        all *= per_seq;
        const int per = share_size(all, (int)gridDim.x);
        const bool planner = share == 0 && wave == 0;
        now = share_begin(all, per, share), end = share_begin(all, per, share + 1);
        if (now >= end && !planner) return;
        // The sequence that holds tile `now`.
        const int want = now / per_seq;  // as tiles of one segment of each sequence
        int before = 0;
        bool found = false;
        for (int q = 0; q < a.batch && (planner || !found); q += kWave) {
            if (a.batch > kWave) group_of(q);
            if (planner && q + lane < a.batch) a.plan[q + lane] = before + upto - own;
            const uint64_t past = __ballot(before + upto > want);
            if (past && !found) {
                found = true;
                const int at = __ffsll((unsigned long long)past) - 1;
                b = q + at;
                len = read_lane(at_len, at), count = read_lane(at_count, at);
                const int rest = now - (before + read_lane(upto - own, at)) * per_seq, each = read_lane(own, at);
                seg = rest / each;
                skip = rest - seg * each;
            }
            before += read_lane(upto, kWave - 1);
        }
        if (planner && lane == 0) a.plan[a.batch] = before, a.plan[a.batch + 1] = per;
        b = uniform(b), seg = uniform(seg), skip = uniform(skip), now = uniform(now), end = uniform(end);
    }

    // 0: the usual one. 1 and 2, where that has met scales beyond kLeastScale and
    // kMostScale: without scales of values, for the rows' maxima and sums; with
    // them, for the output.
    int pass = 0;
    while (now < end) {
    const Arguments A = arguments_again();
    len = uniform(len), count = uniform(count);
    const int total = tokens_of(len, count);
    const int h = seg / A->row_blocks, rb = seg - h * A->row_blocks;
    const int64_t slot = direct ? 0 : share + (int64_t)b * per_seq + seg;
    const int seg_tiles = count > 0 ? (total + TT - 1) / TT : 0;
    // No rows in this block of rows (the nodes it would hold do not exist).
    const bool rows_in = rb * S::kRows < count * group;
    const int mine = direct ? seg_tiles : min(seg_tiles - skip, end - now);
    const int first = skip * TT, last = min(total, first + mine * TT);
    if (rows_in || direct) {

    // The team's tiles are numbered from 0 at `origin`, TT tokens apart. A tile
    // goes through three steps: lookup() asks for the page of a lane's token;
    // settle() notes where the token's rows start; fetch() asks for the rows. A
    // page outside the cache is not followed: its tokens read as zeros, as
    // those from `last` on do. (Two tiles on their way, with twice the
    // registers: 37.9 us / 40.8 in the case above, where nothing spilled.)
    const int origin = first + wt * TS;
    const int32_t* pages = A->table + b * A->table_stride;
    // AT_ONCE tiles at once, a lane a token, by one wave.
    constexpr int AT_ONCE = HELD == 2 ? 1 : kWave / TS;
    const int ahead = AT_ONCE == 1 ? 0 : lane / TS, mine_t = lane % TS;  // this lane's tile of them, and token
    const bool looks = WM == 1 || wm == 0;
    int page = -1, at = 0;
    auto lookup = [&](int i) {
        if (!looks) return;
        const int t = origin + (i + ahead) * TT + mine_t;
        const int number = __umulhi((uint32_t)t << 2, A->places_factor) >> A->places_shift;
        at = t - number * A->cache.places;
        page = t < last ? pages[number] : -1;
    };
    int64_t scale_at = -1;  // of this lane's token in the tiles settled last
    auto settle = [&](int i) {
        if (!looks) return;
        const bool in = page >= 0 && page < A->cache.pages;
        const uint64_t all = __ballot(in);
        const int slot = (i + ahead) % 4;
        offs[slot][mine_t] = in ? (uint32_t)page * A->page16 + (uint32_t)at * A->place16 : 0;
        if (mine_t == 0) held[wt][slot] = TS == 64 ? all : all >> (32 * ahead) & 0xFFFFFFFFu;
        if constexpr (kScaled)
            scale_at = in ? (int64_t)((uint64_t)(uint32_t)page * (uint32_t)A->cache.scale_page_stride + (uint64_t)(uint32_t)at * (uint32_t)A->cache.scale_place_stride) : -1;
    };
    constexpr uint64_t kAllIn = TS == 64 ? ~0ull : 0xFFFFFFFFull;
    const char* const kh = static_cast<const char*>(A->cache.k) + h * A->cache.head_stride * C::kBytes;
    const char* const vh = static_cast<const char*>(A->cache.v) + h * A->cache.head_stride * C::kBytes;
    const float* const ksh = A->cache.k_scales + h * A->cache.scale_head_stride;
    const float* const vsh = A->cache.v_scales + h * A->cache.scale_head_stride;
    u32x4 rk[NL], rv[NL];
    float sk = 0.f, sv = 1.f;
    auto row_at = [&](int j) { return min((j * S::kTeam + tm) / S::kRowLoads, TS - 1); };
    auto column_at = [&](int j) { return (j * S::kTeam + tm) % S::kRowLoads * S::kPerLoad; };
    // Where a team is a wave its loads do not stay in the caches: all rows that
    // read the token are in this block. Where it is the block they do, for the
    // other blocks of rows. (Staying / not: 32 sequences x 32 rows 129 us / 121;
    // 4 sequences x 512 rows 98.6 / 108.6.)
    auto fetch_one = [&](int j, uint32_t off) {
        const int c = column_at(j);
        const uint64_t at = (uint64_t)off * 16 + (c < D ? c : 0) * C::kBytes;
        rk[j] = load_vec<HELD == 1>(reinterpret_cast<const u32x4*>(kh + at));
        rv[j] = load_vec<HELD == 1>(reinterpret_cast<const u32x4*>(vh + at));
    };
    // Of tile i, by the lanes that looked its tokens up.
    auto fetch_scales = [&](int i) {
        if constexpr (kScaled) {
            if (looks && ahead == i % AT_ONCE) {
                sk = 0.f, sv = 1.f;
                if (scale_at >= 0) sk = ksh[scale_at], sv = vsh[scale_at];
            }
        }
    };
    // Infinities and NaN in the values of nodes are left out of the products
    // (0 times them would reach rows that do not see the node) and noted;
    // strange() gives them to the rows that do.
    auto clean = [&](u32x4 v) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            constexpr uint32_t X = Mma<VT>::kExponent;
            const uint32_t keep = ((v[w] & X) == X ? 0u : 0xFFFFu) | ((v[w] >> 16 & X) == X ? 0u : 0xFFFF0000u);
            if (keep != ~0u) atomicOr(&notes, kOdd);
            v[w] &= keep;
        }
        return v;
    };
    auto fetch = [&](int i) {
        uint32_t off[NL];
#pragma unroll
        for (int j = 0; j < NL; ++j) off[j] = offs[i % 4][row_at(j)];
#pragma unroll
        for (int j = 0; j < NL; ++j) fetch_one(j, off[j]);
        fetch_scales(i);
    };
    auto store = [&](int i) {
        char* const ldsk = tiles_lds + i % HELD * S::kTileBytes;
        char* const ldsv = ldsk + TS * S::kPitchK;
        const int base = origin + i * TT;
        const uint64_t in = held[wt][i % 4];
        const bool part = uniform((int)(in != kAllIn)) || DP != D;
        if constexpr (kScaled) {
            if (looks && ahead == i % AT_ONCE) {
                // A scale that is no number (of a row that held an infinity or a NaN)
                // is left out of the weights, which it has no part in, and
                // noted: the rows that see the token get it at the end.
                float c = pass == 1 ? 1.f : sv;
                if (__builtin_expect(!(c >= kLeastScale && c <= kMostScale), false)) {
                    const bool number = c < __builtin_inff();
                    if (c != 0.f) atomicOr(&notes, number ? kBeyond : base + mine_t < len ? kLost : kOdd);
                    c = !number ? 1.f : c != 0.f ? fmaxf(c, 0x1p-100f) : pass ? 0x1p-90f : kZeroScale;
                }
                auto& f = factors[wt][i % HELD];
                f[0][mine_t] = sk * A->scale;
                f[1][mine_t] = __builtin_amdgcn_logf(c);
                f[2][mine_t] = 1.f / c;
            }
        }
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            const int e = j * S::kTeam + tm, t = e / S::kRowLoads, c = e % S::kRowLoads;
            __builtin_amdgcn_sched_barrier(0);  // one row's conversion at a time: registers
            if (NL * S::kTeam == TS * S::kRowLoads || e < TS * S::kRowLoads) {
                if (part && !((in >> t & 1) && c * S::kPerLoad < D)) rk[j] = rv[j] = u32x4{0, 0, 0, 0};
                u32x4* dk = reinterpret_cast<u32x4*>(ldsk + t * S::kPitchK + c * 16);
                u32x4* dv = reinterpret_cast<u32x4*>(ldsv + t * S::kPitchV + c * 16);
                if constexpr (kScaled) {
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const u32x2 k0 = C::template widen4<T>(rk[j][2 * p]), k1 = C::template widen4<T>(rk[j][2 * p + 1]);
                        const u32x2 v0 = C::template widen4<VT>(rv[j][2 * p]), v1 = C::template widen4<VT>(rv[j][2 * p + 1]);
                        dk[p * S::kRowLoads] = u32x4{k0[0], k0[1], k1[0], k1[1]};
                        dv[p * S::kRowLoads] = u32x4{v0[0], v0[1], v1[0], v1[1]};
                    }
                } else {
                    *dk = rk[j];
                    *dv = rv[j];
                }
            }
        }
        if (!std::is_same_v<C, CachedI8> && base + TS > len) {  // what this thread wrote of nodes
#pragma unroll 1
            for (int j = 0; j < NL; ++j) {
                const int e = j * S::kTeam + tm, t = e / S::kRowLoads, c = e % S::kRowLoads;
                if (e >= TS * S::kRowLoads || base + t < len) continue;
                u32x4* dv = reinterpret_cast<u32x4*>(ldsv + t * S::kPitchV + c * 16);
#pragma unroll 1
                for (int p = 0; p < S::kPerLoad / 8; ++p) dv[p * S::kRowLoads] = clean(dv[p * S::kRowLoads]);
            }
        }
    };
    auto team_sync = [&]() {
        if constexpr (WM > 1) __syncthreads();
        else wave_lds_fence();
    };

    const int tiles = rows_in && last > origin ? (last - origin + TT - 1) / TT : 0;
    lookup(0);
    // This lane's row, looked at while the pages are on their way.
    const int row = (rb * WM + wm) * RW + n;
    uint64_t seen;  // the nodes it sees
    u32x4 qf[KS];
    {
        const int node = row / group, g = row - node * group;
        const bool live = row < M && node < count;
        seen = ~0ull >> (63 - min(node, 63));
        if (A->mask) seen = (uint64_t)A->mask[(int64_t)b * A->nodes + (live ? node : 0)];
        seen = live ? seen & (count >= 64 ? ~0ull : (1ull << count) - 1) : 0;
        const uint16_t* q = static_cast<const uint16_t*>(A->q);
        if (live) q += b * A->q_batch + node * A->q_node + (h * group + g) * A->q_head;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int d = S::dim_of(s * KD + part * 8);
            qf[s] = *reinterpret_cast<const u32x4*>(q + (d < D ? d : 0));
            qf[s] = (qf[s] ^ A->flip) & (live && d < D ? A->keep : 0u);
        }
    }

    __syncthreads();  // the segment before is done with the LDS
    if (tid == 0) notes = 0;
    settle(0);
    __syncthreads();
    if (tiles > 0) fetch(0);
    Acc o[DT];
    float m = -__builtin_inff(), l = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = Acc{};

    if constexpr (HELD == 2) {
        lookup(1);
        settle(1);
        if (tiles > 0) store(0);
        lookup(2);
        __syncthreads();
        if (tiles > 1) fetch(1);
        settle(2);
        __syncthreads();
    }
    for (int i = 0; i < tiles; ++i) {
        const int base = origin + i * TT;
        // With one tile in the LDS it is written before its products, with
        // two the next is written beside them. The pages of tiles to come are
        // looked up here and settled at the end, before they are fetched in
        // the next turn; by a team of one wave after it has its rows, since it
        // would wait for the pages as well (32 sequences x 32 rows, int8: 121
        // us / 115.5; the block's first wave alone looks, and that costs it
        // nothing that the order would save).
        const bool look = HELD == 2 || i % 2 == 0;
        constexpr int TO_COME = HELD == 2 ? 3 : 2;
        if constexpr (HELD == 2) lookup(i + TO_COME);
        if constexpr (HELD == 1) {
            wave_lds_fence();
            store(i);
            wave_lds_fence();
            if (look) lookup(i + TO_COME);
            if (i + 1 < tiles) fetch(i + 1);
        }
        const char* const ldsk = tiles_lds + i % HELD * S::kTileBytes;
        const char* const ldsv = ldsk + TS * S::kPitchK;
        auto& kfac = factors[wt][i % HELD][0];
        auto& vlog = factors[wt][i % HELD][1];
        auto& vinv = factors[wt][i % HELD][2];

        // Scores of this wave's tokens.
        Acc sc[SUB * X / OX];  // OX values each
#pragma unroll
        for (int s = 0; s < SUB * X / OX; ++s) {
            sc[s] = Acc{};
            const char* kp = ldsk + (s * RW + n) * S::kPitchK + part * 16;
#pragma unroll
            for (int k = 0; k < KS; ++k) sc[s] = Mma<T>::dot(*reinterpret_cast<const u32x4*>(kp + k * KD * 2), qf[k], sc[s]);
        }
        // Value x of 32 tokens.
        auto score = [&](int s, int x) -> auto& { return sc[(s * X + x) / OX]; };
        if constexpr (HELD == 2) {
            if (i + 1 < tiles) store(i + 1);
            if (i + 2 < tiles) fetch(i + 2);
        }
        if constexpr (kScaled) {
#pragma unroll
            for (int s = 0; s < SUB; ++s)
#pragma unroll
                for (int x = 0; x < X; x += 4) {
                    const int t = s * 32 + PARTS * x + 4 * part;
                    const f32x4 kf = *reinterpret_cast<const f32x4*>(kfac + t), vl = *reinterpret_cast<const f32x4*>(vlog + t);
#pragma unroll
                    for (int y = 0; y < 4; ++y) score(s, x)[(x + y) % OX] = score(s, x)[(x + y) % OX] * kf[y] + vl[y];
                }
        }
        if (base + TS > min(len, total)) {
            // Bit t of a word: whether this lane's row sees token t of 32.
#pragma unroll
            for (int s = 0; s < SUB; ++s) {
                const int from = base + s * 32, j = from - len, left = total - from;
                const uint32_t there = left >= 32 ? ~0u : left > 0 ? (1u << left) - 1 : 0u;
                uint32_t sees = j <= -32 ? ~0u : j >= 64 ? 0u : j >= 0 ? (uint32_t)(seen >> j) : (uint32_t)(seen << -j) | ((1u << -j) - 1);
                sees = (sees & there) >> (4 * part);
#pragma unroll
                for (int x = 0; x < X; ++x)
                    if (!(sees & 1u << (4 * PARTS * (x / 4) + x % 4))) score(s, x)[x % OX] = -__builtin_inff();
            }
        }
        float top4[4] = {-__builtin_inff(), -__builtin_inff(), -__builtin_inff(), -__builtin_inff()};
#pragma unroll
        for (int s = 0; s < SUB; ++s)
#pragma unroll
            for (int x = 0; x < X; ++x) top4[x % 4] = fmaxf(top4[x % 4], score(s, x)[x % OX]);
        float top = join_parts<PARTS>(fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3])), [](float x, float y) { return fmaxf(x, y); });
        if constexpr (!kScaled) top *= A->scale;
        if (__any(top > m + kLazy)) {
            const float to = top > m + kLazy ? top : m;
            const float f = to == m ? 1.f : __builtin_amdgcn_exp2f(m - to);
            m = to;
            l *= f;
#pragma unroll
            for (int d = 0; d < DT; ++d) o[d] *= f;
        }
        const float ms = m == -__builtin_inff() ? 0.f : m;
        uint32_t pf[SUB][X / 2];
#pragma unroll
        for (int s = 0; s < SUB; ++s) {
#pragma unroll
            for (int x = 0; x < X; x += 4) {
                f32x4 vi;
                if constexpr (kScaled) vi = *reinterpret_cast<const f32x4*>(vinv + s * 32 + PARTS * x + 4 * part);
                float w[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const float v = score(s, x)[(x + y) % OX];
                    w[y] = __builtin_amdgcn_exp2f(kScaled ? v - ms : v * A->scale - ms);
                    l += kScaled ? w[y] * vi[y] : w[y];
                }
                pf[s][x / 2] = Mma<VT>::pack(w[0], w[1]);
                pf[s][x / 2 + 1] = Mma<VT>::pack(w[2], w[3]);
            }
        }
        // 8 tokens of a column, those of values 8k .. 8k + 7: 16 lanes read 4
        // tokens times 16 columns, twice; lane % 16 picks a column.
        auto values = [&](int s, int k, int d) -> u32x4 {
            const char* vp = ldsv + (s * 32 + k * 8 * PARTS + 4 * part + (lane % 16) / 4) * S::kPitchV +
                             (lane % RW / 16) * 32 + (lane % 4) * 8 + d * RW * 2;
            using L = __attribute__((address_space(3))) s16x4*;
            const u32x2 v0 = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((L)vp));
            const u32x2 v1 = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((L)(vp + 4 * PARTS * S::kPitchV)));
            return u32x4{v0[0], v0[1], v1[0], v1[1]};
        };
#pragma unroll
        for (int s = 0; s < SUB; ++s)
#pragma unroll
            for (int k = 0; k < X / 8; ++k)
#pragma unroll
                for (int d = 0; d < DT; ++d)
                    o[d] = Mma<VT>::dot(values(s, k, d), u32x4{pf[s][4 * k], pf[s][4 * k + 1], pf[s][4 * k + 2], pf[s][4 * k + 3]}, o[d]);
        if (look) settle(i + TO_COME);
        team_sync();
    }

    const Arguments E = arguments_again();
    // Where a row's sums go: to the output, or to the partials of this chunk.
    const int64_t prow0 = slot * S::kRows - rb * S::kRows;
    auto out_of = [&](int rw) {
        const int node = rw / group, g = rw - node * group;
        return static_cast<uint16_t*>(E->out) + b * E->out_batch + node * E->out_node + (h * group + g) * E->out_head;
    };
    auto put_stats = [&](int rw, float mm, float ll) {
        if (direct) {
            const int node = rw / group, g = rw - node * group;
            if (node >= count) ll = 0.f;
            E->lse[((int64_t)b * E->nodes + node) * (heads * group) + h * group + g] =
                ll > 0.f || ll != ll ? (mm + __builtin_amdgcn_logf(ll)) * 0.69314718055994531f : -__builtin_inff();
        } else {
            E->part_ml[prow0 + rw] = make_float2(mm, ll);
        }
    };
    // The infinities and NaN in columns c .. c + 3 of the nodes of this chunk
    // that row rw sees: their weights do not matter. All columns are NaN where
    // a scale that it sees is no number.
    auto strange = [&](int rw, int c) {
        constexpr float kNaN = __builtin_nanf("");
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        const int node = rw / group;
        if (node >= count) return v;
        if (notes & kLost) return f32x4{kNaN, kNaN, kNaN, kNaN};
        const uint64_t word = E->mask ? (uint64_t)E->mask[(int64_t)b * E->nodes + node] : ~0ull >> (63 - node);
#pragma unroll 1
        for (int t = max(first, len); t < last; ++t) {
            const int page = E->table[b * E->table_stride + t / E->cache.places];
            if (!(word >> (t - len) & 1) || page < 0 || page >= E->cache.pages) continue;
            if constexpr (kScaled) {
                const int64_t of = (int64_t)page * E->cache.scale_page_stride + (int64_t)(t % E->cache.places) * E->cache.scale_place_stride + h * E->cache.scale_head_stride;
                if (!(E->cache.v_scales[of] < __builtin_inff())) return f32x4{kNaN, kNaN, kNaN, kNaN};
            }
            const int64_t at = (int64_t)page * E->cache.page_stride + (int64_t)(t % E->cache.places) * E->cache.place_stride + h * E->cache.head_stride + c;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                float f;
                if constexpr (kScaled)
                    f = F16::widen((uint16_t)C::template widen4<F16>(static_cast<const uint8_t*>(E->cache.v)[at + y])[0]);
                else
                    f = T::widen(static_cast<const uint16_t*>(E->cache.v)[at + y]);
                if (!(__builtin_fabsf(f) < __builtin_inff())) v[y] += f;
            }
        }
        return v;
    };
    auto put4 = [&](int rw, int c, f32x4 v, float ll) {
        if (direct) {
            const float inv = ll > 0.f || ll != ll ? 1.f / ll : 0.f;
            u32x2 w = {Mma<T>::pack(v[0] * inv, v[1] * inv), Mma<T>::pack(v[2] * inv, v[3] * inv)};
            if (ll == 0.f || rw >= count * group) w = u32x2{0, 0};
            *reinterpret_cast<u32x2*>(out_of(rw) + c) = w;
        } else {
            *reinterpret_cast<f32x4*>(E->part_o + (prow0 + rw) * D + c) = v;
        }
    };
    // The sum of row r of the block, found with the maximum mm: in pass 2 that of
    // pass 1, brought to this pass's maximum in two halves (its own may be as far
    // away as the scales are apart).
    auto settled = [&](int r, float mm, float ll, bool first) {
        if constexpr (kScaled) {
            if (pass == 1 && first) unscaled[0][r] = mm, unscaled[1][r] = ll;
            if (pass == 2) {
                const float half = __builtin_amdgcn_exp2f(0.5f * (unscaled[0][r] - mm));
                ll = unscaled[1][r] == 0.f ? 0.f : unscaled[1][r] * half * half;
            }
        }
        return ll;
    };
    float ll = join_parts<PARTS>(l, [](float x, float y) { return x + y; });
    // Columns of an accumulator, in fours: 4 PARTS (y / 4) + 4 part.
    if constexpr (WT == 1) {
        if (row < M) {
            ll = settled(wm * RW + n, m, ll, part == 0);
            if (part == 0) put_stats(row, m, ll);
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int y = 0; y < OX; y += 4) {
                    const int c = S::dim_of(d * RW + PARTS * y + 4 * part);
                    if (c < D) put4(row, c, f32x4{o[d][y], o[d][y + 1], o[d][y + 2], o[d][y + 3]}, ll);
                }
        }
    } else {
        if (part == 0) red[0][wave][n] = m;
        __syncthreads();
        float mm = -__builtin_inff();
#pragma unroll
        for (int w = 0; w < WT; ++w) mm = fmaxf(mm, red[0][w][n]);
        const float f = m == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(m - mm);
        if (part == 0) red[1][wave][n] = ll * f;
        float* ob = reinterpret_cast<float*>(tile) + (wave * RW + n) * S::kPitchO;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int y = 0; y < OX; y += 4)
                *reinterpret_cast<f32x4*>(ob + S::dim_of(d * RW + PARTS * y + 4 * part)) = f32x4{o[d][y], o[d][y + 1], o[d][y + 2], o[d][y + 3]} * f;
        __syncthreads();
        for (int e = tid; e < RW * (DP / 4); e += S::kThreads) {
            const int rn = e / (DP / 4), c = e % (DP / 4) * 4, rw = rb * S::kRows + rn;
            if (c >= D || rw >= M) continue;
            f32x4 v = {0.f, 0.f, 0.f, 0.f};
            float lsum = 0.f, mx = -__builtin_inff();
#pragma unroll
            for (int w = 0; w < WT; ++w) {
                v += *reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(tile) + (w * RW + rn) * S::kPitchO + c);
                lsum += red[1][w][rn];
                mx = fmaxf(mx, red[0][w][rn]);
            }
            lsum = settled(rn, mx, lsum, c == 0);
            if (c == 0) put_stats(rw, mx, lsum);
            put4(rw, c, v, lsum);
        }
    }
    __syncthreads();
    if (notes & (kOdd | kLost)) {
        for (int e = tid; e < S::kRows * (DP / 4); e += S::kThreads) {
            const int c = e % (DP / 4) * 4, rw = rb * S::kRows + e / (DP / 4);
            if (c >= D || rw >= M) continue;
            const f32x4 v = strange(rw, c);
            for (int y = 0; y < 4; ++y) {
                if (v[y] == 0.f) continue;
                if (direct) out_of(rw)[c + y] = T::narrow(v[y]);
                else E->part_o[(prow0 + rw) * D + c + y] = v[y];
            }
        }
    }
    if (kScaled && (pass ? pass == 1 : (notes & kBeyond) != 0)) {
        ++pass;
        continue;
    }
    }
    pass = 0;
    now += direct ? 1 : mine;
    skip = 0;
    if (now < end) {  // the next segment that has tiles
        do {
            if (++seg == per_seq) {
                seg = 0, ++b;
                load_sequence(b, &len, &count);
                len = uniform(len), count = uniform(count);
            }
        } while (count == 0 || tokens_of(len, count) == 0);
    }
    }
}

template <class T, class C, int DP, int RW, int WM, int WT, int TS>
hipError_t launch_attention_shape(const TreeAttention& a, hipStream_t stream) {
    const unsigned int grid = a.blocks ? (unsigned)a.blocks : (unsigned)(a.batch * a.cache.heads * a.row_blocks);
    tree_attention_kernel<T, C, DP, RW, WM, WT, TS><<<grid, kWave * WM * WT, 0, stream>>>(a);
    return hipGetLastError();
}

template <class T, class C, int DP>
hipError_t launch_attention_dim(const TreeAttention& a, hipStream_t stream) {
    const int rows = a.nodes * a.group;
    const AttentionShape s = attention_shape(rows, DP, C::kBytes);
    if (s.is(kFewestRows)) return launch_attention_shape<T, C, DP, 16, 1, 4, 32>(a, stream);
    if (s.is(kHalfRows)) return launch_attention_shape<T, C, DP, 16, 4, 1, 32>(a, stream);
    if constexpr (DP <= kNarrowHeads) {
        if constexpr (C::kBytes == 1 || DP <= kNarrowPairs)
            if (s.is(kFewRows)) return launch_attention_shape<T, C, DP, 32, 1, 4, 32>(a, stream);
        return launch_attention_shape<T, C, DP, 32, 4, 1, 64>(a, stream);
    }
    return hipErrorInvalidValue;  // not reached: the shapes above are all that wide heads take
}

template <class T, class C>
hipError_t launch_attention(const TreeAttention& a, hipStream_t stream) {
    const int d = a.cache.dim;
    if (d <= 64) return launch_attention_dim<T, C, 64>(a, stream);
    if (d <= 96) return launch_attention_dim<T, C, 96>(a, stream);
    if (d <= 128) return launch_attention_dim<T, C, 128>(a, stream);
    if (d <= 192) return launch_attention_dim<T, C, 192>(a, stream);
    return launch_attention_dim<T, C, 256>(a, stream);
}

}  // namespace libred
