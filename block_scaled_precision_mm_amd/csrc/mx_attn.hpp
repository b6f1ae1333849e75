// mx_attn.hpp -- attention of each sequence's new tokens over the paged MX
// key/value cache (mx_cache.hpp), gfx950.
//
// For query row (token, head) of a sequence with n new tokens and L keys, the
// token at position pos = L - n + i:
//     x_j  = scale * q . k_j          over the keys j it sees
//     out  = sum_j exp(x_j) v_j / sum_j exp(x_j),   lse = log sum_j exp(x_j)
// in one pass over the keys with a running maximum: the sums are kept
// relative to a reference m, p_j = 2^(x_j log2 e - m).  A row that sees no key
// gives 0 and lse = -inf.
//
// Types.  Codes are expanded to BF16 on the way into LDS (exactly within its
// range: an E4M3 or E2M1 element times a power of two has at most 4
// significant bits), both products run on the BF16 MFMA with FP32
// accumulation, q.k of the given BF16 q is exact but for the accumulation, x,
// m and the sums are FP32.  p is rounded to BF16 as the second product's
// operand (half a step: 2^-8 of each p): values need BF16's range (FP16 would
// lose a block whose scale is far from the others'), and a BF16 output is
// rounded as coarsely itself: over a call's outputs it is off by 0.0020 to
// 0.0023 of them, 2-norms, where its own rounding makes 0.0017.  The sum of the
// p's takes them unrounded.
//
// Trees (P2) take p in two parts, BF16(p) and BF16 of the rest, with a second
// MFMA each, within 2^-16 of each p: for FP16 and FP32 outputs, which are then
// off by 2e-6 in FP32 instead of 0.0011 to 0.0016, and in tiles of 16 rows for
// BF16 ones too.  There loads and joins are what bounds a call, and so few rows
// do not average what a p is off by (one row over 7728 keys 0.0028).  us with one
// part and with two, tiles of 16 rows: 27 nodes over 1051 keys 12.8 and 12.95, 32
// sequences of 4 over 4096 57.6 and 57.8, 64 of 2 over 8000 in E2M1 102 and 106.
// The tiles of more rows: 32 ragged trees 75 and 80, 24 under a window 24.1 and
// 26.4, two over 131072 and 80868 keys, where MFMAs bound it, 400 and 538.
//
// The rows of one KV head.  All G = q_heads / kv_heads query heads of a KV
// head read the same keys, so a tile's rows are (token, head of the group)
// pairs, token-major: keys are read and expanded once for the group, and a
// short chunk fills the MFMA's rows with heads.
//
// Transposed products.  S^T = K Q^T and O^T = V^T P^T: a lane of the
// accumulators holds one query row and several keys, so the softmax runs
// inside lanes plus an exchange between the lanes of a row, rescaling O is a
// multiplication by a lane's own factor, and P^T is already in the layout
// of the second product's operand: the contraction over keys may take them
// in any order, and V^T is read in the order in which S^T left them (two
// transposing LDS reads of four keys each).
//
// Rescaling.  The p of a tile are taken under the reference so far, and m is
// raised to the row's maximum only where their sum passes 4096 (a wave-uniform
// branch that also catches the first tile, where m = -inf makes them infinite
// or NaN): until then FP32 sums and BF16's relative precision do not notice,
// and the maximum of a tile need not be found (24 of 115 VALU instructions).
//
// Work (plan_item).  Sequence lengths are known on the device only.  A launch
// has as many workgroups as can run at once plus one per (sequence, head,
// row tile); each finds its own item from the lengths: key ranges longer
// than the average work per resident workgroup are split, and the parts of
// one row tile joined through a workspace, by the workgroup that arrives
// last (few rows) or by a second kernel (many rows), in a fixed order, so
// results do not depend on timing.
//
// Trees of drafted tokens (TREE).  The rows of a sequence see its whole context
// and of the new keys, its nodes, those of their mask's bits.  So only tiles
// that hold a node, the last of a sequence, look at masks: a word or two per
// row and tile, in the branch that other partly seen tiles take; the rest is
// the same loop.  Bound as it: one tree of 27 nodes over 1051 keys 12.9 us (the
// chain of dependent loads and the join of the parts), 32 of 16 over 100 to
// 16000 keys, 64 rows a KV head, 75 to 78 us (239 MB, 3.1 TB/s; every key is
// expanded for two row tiles: VALU busy for 35% and MFMA for 16% of the SIMDs'
// cycles, and 68% of the two waves that a SIMD has room for there, as items are
// unequal), two of 488 and 344 rows over 131072 and 80868 keys in E2M1 387 to 415
// us (0.91 to 0.97 PFLOP/s; VALU 42%, MFMA 49%).  A tree's launch has one kernel
// for all rows; its parts are chosen so that items run at once (one_round), as
// there are too few rows for many rounds.
//
// Masked places.  Scores of unseen keys are replaced, never added to;
// values of slots past the sequence's end or on pages outside the cache are
// replaced by zeros as they are expanded.  A NaN or infinity (a code under a
// scale that takes it past BF16's range) among the values of a key that some
// rows of a tile see and others do not would reach the others as 0 * NaN or
// 0 * inf: in tiles that not every row sees whole they become zeros as they
// are expanded.  Where there was one, or a sum is not finite at the end
// (rare), the item's keys are looked through once more and the rows that see
// one get it from the codes themselves (attn_special): a sum that sees an
// infinity is that infinity whatever its weight, one that sees a NaN or both
// infinities is NaN.
#pragma once

#include <type_traits>

#include "mx_cache.hpp"
#include "mx_splitk.hpp"
#include "mx_sync.hpp"

namespace mxg {

typedef float v16f __attribute__((ext_vector_type(16)));

// Compile-time loop: f(IntC<B>) for B in [B0, B1).
template <int N> struct IntC { static constexpr int value = N; };
template <int B0, int B1, class Fn>
__device__ __forceinline__ void static_range(Fn &&f)
{
    if constexpr (B0 < B1) {
        f(IntC<B0>{});
        static_range<B0 + 1, B1>(f);
    }
}

typedef __bf16 bf16x8v __attribute__((ext_vector_type(8)));
typedef short s16x4v __attribute__((ext_vector_type(4)));

struct AttnArgs {
    const uint8_t *codes[2], *scales[2];    // keys, values
    const uint16_t *q;                      // [tokens][q_heads][dim], q_stride elements between tokens
    const int *ends, *lens, *table;
    void *out;                              // [tokens][q_heads][dim]
    float *lse;                             // [tokens][q_heads] or null
    unsigned *counters;                     // one per row tile; null: no splitting
    uint8_t *parts;                         // partial results of split row tiles
    long long q_stride, table_stride;
    float c;                                // scale * log2 e
    int seqs, tokens, heads, group;         // KV heads, query heads per KV head
    FastDiv by_heads, by_group;
    int page_shift, pages, table_width;
    int causal, window;
    int out_kind;
    int rows_above, rows_upto;              // the sequences of this launch: rows_above < n * group <= rows_upto
    float per_target;                       // KV heads / workgroups that can run at once
    const unsigned long long *mask;         // trees of drafted tokens: [tokens][mask_words], the nodes that each sees
    int mask_words;
    int resident;                           // (trees) workgroups that can run at once
};

// One workgroup's work.
struct AttnItem {
    int seq, head, tok0, ntok, len;         // first row of q, new tokens, keys
    int row0;                               // first row of the tile among ntok * group
    int key0, key1;                         // its keys (key0 a multiple of BN)
    int all_lo, all_hi;                     // keys that every row of the tile sees
    int part, parts, slot, slot_step;       // split row tiles: this part, their number, workspace slots
    int counter;
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A wave-uniform v that the compiler knows nothing about: in a loop, addresses
// made from it are computed where they are used, and not kept in registers
// that are stepped beside it (mx_attn_tile: 18 registers in scratch memory and
// 4096 tokens behind 12204 keys in 926 us, otherwise 825).
__device__ __forceinline__ int opaque(int v)
{
    asm("" : "+s"(v));
    return v;
}

// Inclusive sums over the wave's lanes (DPP row shifts and broadcasts).
template <class T, int CTRL, int ROWS>
__device__ __forceinline__ T dpp_or_0(T v)
{
    return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xF, false));
}

template <class T>
__device__ __forceinline__ T wave_prefix(T v)
{
    v += dpp_or_0<T, 0x111, 0xF>(v);
    v += dpp_or_0<T, 0x112, 0xF>(v);
    v += dpp_or_0<T, 0x114, 0xF>(v);
    v += dpp_or_0<T, 0x118, 0xF>(v);
    v += dpp_or_0<T, 0x142, 0xA>(v);
    v += dpp_or_0<T, 0x143, 0xC>(v);
    return v;
}

__device__ __forceinline__ int lane_value(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

// v of the lane before; `first` in lane 0.
__device__ __forceinline__ int lane_before(int v, int first)
{
    return __builtin_amdgcn_update_dpp(first, v, 0x138, 0xF, 0xF, false);
}

// A sequence as a lane sees it: row tiles and key tiles of the sequences of
// this launch's class, 0 row tiles for others.
struct AttnSeq {
    int tok0, ntok, len, rtiles, ktiles;
};

// carry: the end of the sequences before s - lane, updated to that of the 64.
// Ends are taken as min(tokens, max(0, ends[0 .. s])), as group ends are
// (mx_group.hpp), so the sequences' rows never overlap whatever they hold.
template <int BM, int BN>
__device__ __forceinline__ AttnSeq attn_seq(const AttnArgs &p, int s, int &carry)
{
    const int lane = threadIdx.x & 63;
    AttnSeq q = {0, 0, 0, 0, 0};
    int end = carry;
    const bool mine = s < p.seqs;
    if (mine) {
        end = min(max(p.ends[s], carry), p.tokens);
        q.len = min(max(p.lens[s], 0), p.table_width << p.page_shift);
    }
    int before = lane_before(end, carry);
    if (__any(mine && end < before)) {
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int u = __shfl_up(end, d);
            end = lane >= d ? max(end, u) : end;
        }
        before = lane_before(end, carry);
    }
    carry = lane_value(end, 63);
    q.tok0 = before;
    q.ntok = mine ? end - before : 0;
    const int rows = q.ntok * p.group;
    if (rows > p.rows_above && rows <= p.rows_upto) {
        q.rtiles = (rows + BM - 1) / BM;
        // (with a window the keys before the first token's are not read)
        const int lo = p.window > 0 ? max(0, q.len - q.ntok - p.window + 1) : 0;
        q.ktiles = (q.len + BN - 1) / BN - min(lo, q.len) / BN;
    }
    return q;
}

__device__ __forceinline__ int cdiv_u(int a, int b) { return (int)(((unsigned)a + (unsigned)b - 1u) / (unsigned)b); }

// Trees: the smallest chunk, from `least` on, with which all items run at
// once.  (Chunks of the average work make up to one item per row tile more
// than run at once, and those few are a second round: two sequences of 61 and
// 43 nodes over 131072 and 80868 keys, 272 items of 256 rows for 256
// workgroups, took 650 us, and in one round 400.)  Where the row tiles alone are
// too many for that, or it would leave the workgroups half idle: the average
// work, which cuts none of like sequences, or 1.3 times that where some sequence
// has far more: there the long ones' items go first (plan_item), so that short
// ones fill the end (32 sequences of 100 to 16000 keys 77 us; with the average
// work 89, twice that 83, half of it in the sequences' order 92).  More than 64
// sequences, which a wave does not hold at once, have the average work and
// their own order: 64 such sequences 141 us, 65 155, 128 285 (0.45, 0.45 and 0.91 GB).
__device__ __forceinline__ int one_round(const AttnArgs &p, const AttnSeq &q, float total, int least)
{
    if (p.seqs > 64)
        return least;
    const int rounds = __any(q.ktiles > 2 * least) ? (int)(1.3f * (float)least) : least;
    const int last = p.seqs > 1 ? 63 : 0;
    int tiles = p.heads * q.rtiles;
    if (p.seqs > 1)
        tiles = wave_prefix(tiles);
    tiles = lane_value(tiles, last);
    if (tiles == 0 || tiles >= p.resident)
        return rounds;
    const float even = total * (float)p.heads / (float)p.resident;
    int a = max(uniform((int)fminf(even, 1e9f)), least);
    int b = max(uniform((int)fminf(total * (float)p.heads / (float)(p.resident - tiles), 1e9f)) + 2, a);
    for (int i = 0; a < b && i < 8; ++i) {
        const int c = (a + b) >> 1;
        int items = p.heads * q.rtiles * max(1, cdiv_u(q.ktiles, c));
        if (p.seqs > 1)
            items = wave_prefix(items);
        if (lane_value(items, last) <= p.resident)
            b = c;
        else
            a = c + 1;
    }
    return (float)b <= 1.7f * even ? b : rounds;
}

// Find item `item` of the launch; false if there is none.  Every wave of the
// workgroup computes it (all results are wave-uniform).  min_tiles: the
// fewest key tiles worth a part of their own.  JOIN: one item per row tile
// of more than one part (at most as many as there are workgroups to run at
// once), instead of one per part.
//
// A sequence's key tiles are cut into parts of at most `chunk`, where chunk
// is at least the total of (row tile, key tile) pairs over the number of
// workgroups that can run at once: split row tiles then have fewer than
// twice that number of parts in all, which bounds the workspace, and the
// items are at most one per row tile and that number more, which bounds the
// grid (the factor keeps both with the FP32 total's rounding).
template <int TREE, int BM, int BN, int JOIN = 0>
__device__ __forceinline__ bool plan_item(const AttnArgs &p, int item, int min_tiles, AttnItem &it)
{
    const int lane = threadIdx.x & 63;
    int chunk = 1 << 30, carry = 0;
    AttnSeq q = attn_seq<BM, BN>(p, lane, carry);
    const int carry64 = carry;
    if (p.counters) {
        float total = (float)q.rtiles * (float)q.ktiles;
        for (int s0 = 64; s0 < p.seqs; s0 += 64) {
            const AttnSeq r = attn_seq<BM, BN>(p, s0 + lane, carry);
            total += (float)r.rtiles * (float)r.ktiles;
        }
        if (p.seqs > 1)
            total = wave_prefix(total);
        total = __int_as_float(lane_value(__float_as_int(total), p.seqs > 1 ? 63 : 0));
        chunk = max(uniform((int)fminf(total * p.per_target * 1.001f, 1e9f) + 1), min_tiles);
        if constexpr (TREE)
            chunk = one_round(p, q, total, chunk);
    }
    carry = carry64;
    int slots = 0, tiles = 0;                         // before the 64 sequences looked at
    for (int s0 = 0;; s0 += 64) {
        if (s0 >= p.seqs)
            return false;
        if (s0 > 0)
            q = attn_seq<BM, BN>(p, s0 + lane, carry);
        const int parts = max(1, cdiv_u(q.ktiles, chunk));
        const int mytiles = p.heads * q.rtiles, myparts = mytiles * parts, mine = !JOIN ? myparts : parts > 1 ? mytiles : 0;
        int upto = mine, slots_upto = parts > 1 ? myparts : 0, tiles_upto = mytiles;
        if (p.seqs > 1) {
            upto = wave_prefix(upto);
            if (p.counters) {
                slots_upto = wave_prefix(slots_upto);
                tiles_upto = wave_prefix(tiles_upto);
            }
        }
        int owned = mine;
        if (TREE && !JOIN && p.seqs > 1 && p.seqs <= 64) {
            // the items of sequences of long parts first
            const bool is_long = 2 * q.ktiles >= chunk;
            owned = is_long ? mine : 0;
            upto = wave_prefix(owned);
            const int longs = lane_value(upto, 63);
            if (item >= longs) {
                item -= longs;
                owned = is_long ? 0 : mine;
                upto = wave_prefix(owned);
            }
        }
        const int all = lane_value(upto, p.seqs > 1 ? 63 : 0);
        if (item >= all) {
            item -= all;
            if (p.seqs == 1)
                return false;
            slots += lane_value(slots_upto, 63);
            tiles += lane_value(tiles_upto, 63);
            continue;
        }
        const int at = __ffsll((unsigned long long)__ballot(item < upto)) - 1;
        it.seq = s0 + at;
        it.tok0 = lane_value(q.tok0, at);
        it.ntok = lane_value(q.ntok, at);
        it.len = lane_value(q.len, at);
        const int rtiles = lane_value(q.rtiles, at), sparts = lane_value(parts, at), smine = lane_value(owned, at);
        item -= lane_value(upto, at) - smine;
        slots += lane_value(slots_upto, at) - (sparts > 1 ? lane_value(myparts, at) : 0);
        tiles += lane_value(tiles_upto, at) - p.heads * rtiles;
        // heads innermost: the workgroups of a head, which share its keys,
        // are then apart by the number of heads and (with 8) on one XCD
        const int rest = p.by_heads.div(item);
        it.head = item - rest * p.heads;
        it.part = rtiles == 1 ? rest : (int)((unsigned)rest / (unsigned)rtiles);
        // the last row tiles of a causal chunk see the most keys: first
        const int rt = rtiles - 1 - (rest - it.part * rtiles);
        it.row0 = rt * BM;
        it.counter = tiles + rt * p.heads + it.head;
        it.slot = slots + rt * p.heads + it.head;
        it.slot_step = rtiles * p.heads;
        // the keys that some row of the tile sees, and those that all do
        const int t0 = p.by_group.div(it.row0), t1 = min(p.by_group.div(it.row0 + BM - 1), it.ntok - 1);
        // (a tree's rows: the keys of the context, whatever their masks and depths)
        const int pos0 = it.len - it.ntok + (TREE ? 0 : t0), pos1 = TREE ? it.len - 1 : it.len - it.ntok + t1;
        const int hi = !TREE && p.causal ? min(max(pos1 + 1, 0), it.len) : it.len;
        const int lo = p.window > 0 ? min(max(pos0 - p.window + 1, 0), hi) : 0;
        it.all_lo = p.window > 0 ? max(pos1 - p.window + 1, 0) : 0;
        it.all_hi = TREE ? max(pos0, 0) : p.causal ? min(max(pos0 + 1, 0), it.len) : it.len;
        const int k0 = lo / BN, nt = (hi + BN - 1) / BN - k0;
        it.parts = sparts == 1 ? 1 : min(sparts, max(1, cdiv_u(nt, chunk)));
        if (it.part >= it.parts)
            return false;
        it.key0 = k0 * BN;
        it.key1 = hi;
        if (it.parts > 1) {
            const int each = (int)((unsigned)nt / (unsigned)it.parts), more = nt - each * it.parts;
            const int first = each * it.part + min(it.part, more);
            it.key0 = (k0 + first) * BN;
            it.key1 = min(hi, it.key0 + (each + (it.part < more)) * BN);
        }
        return true;
    }
}

// Bits [lo, hi) of 64.
__device__ __forceinline__ unsigned long long bit_range(int lo, int hi)
{
    const unsigned long long from = lo <= 0 ? ~0ull : lo >= 64 ? 0ull : ~0ull << lo;
    const unsigned long long upto = hi >= 64 ? ~0ull : hi <= 0 ? 0ull : ~(~0ull << hi);
    return from & upto;
}

// What one query row sees: keys [lo, hi), and of a tree of drafted tokens
// (TREE) the context's keys [lo, context) and the nodes, keys context + j, of
// its bits.
template <int TREE>
struct AttnRow {
    int lo, hi;
    int token, head;        // token of the sequence, head of the group; token < 0: no such row
};

template <>
struct AttnRow<1> {
    int lo, hi;
    int token, head;
    int context;            // keys before the first node; < 0: nodes of keys before the sequence's first
    const unsigned long long *bits;
};

template <int TREE>
__device__ __forceinline__ AttnRow<TREE> attn_row(const AttnArgs &p, const AttnItem &it, int row)
{
    AttnRow<TREE> r;
    const int token = p.by_group.div(row);
    r.head = row - token * p.group;
    r.token = token < it.ntok ? token : -1;
    if constexpr (TREE) {
        r.hi = token < it.ntok ? it.len : 0;
        r.lo = 0;
        r.context = it.len - it.ntok;
        r.bits = p.mask + (long long)(it.tok0 + max(r.token, 0)) * p.mask_words;
        if (p.window > 0) {
            // the node's depth: the nodes that it sees, but for itself
            int seen = 0;
            for (int w = 0; w < p.mask_words && 64 * w < it.ntok; ++w)
                seen += __popcll(r.bits[w] & (it.ntok - 64 * w >= 64 ? ~0ull : ~(~0ull << (it.ntok - 64 * w))));
            r.lo = min(max(r.context + max(seen - 1, 0) - p.window + 1, 0), max(r.context, 0));
        }
    } else {
        const int pos = it.len - it.ntok + token;
        r.hi = token < it.ntok ? (p.causal ? min(max(pos + 1, 0), it.len) : it.len) : 0;
        r.lo = p.window > 0 ? max(pos - p.window + 1, 0) : 0;
    }
    return r;
}

// The keys key .. key + 63 that a row sees, as bits.
template <int TREE>
__device__ __forceinline__ unsigned long long attn_sees(const AttnArgs &p, const AttnRow<TREE> &row, int key)
{
    if constexpr (TREE) {
        unsigned long long see = bit_range(row.lo - key, min(row.context, row.hi) - key);
        const int node = key - row.context;         // of the first key
        if (node > -64) {
            // (whole words; bits past the last word are zeros)
            const int w = node >> 6, s = node & 63;
            const unsigned long long a = (unsigned)w < (unsigned)p.mask_words ? row.bits[w] : 0ull;
            const unsigned long long b = (unsigned)(w + 1) < (unsigned)p.mask_words ? row.bits[w + 1] : 0ull;
            see |= (s ? a >> s | b << (64 - s) : a) & bit_range(row.context - key, row.hi - key);
        }
        return see;
    } else {
        return bit_range(row.lo - key, row.hi - key);
    }
}

// Whether it sees key k.
template <int TREE>
__device__ __forceinline__ bool attn_sees_key(const AttnArgs &p, const AttnRow<TREE> &row, int k)
{
    if constexpr (TREE) {
        const int node = k - row.context;
        if (node < 0)
            return k >= row.lo && k < row.hi;
        return k < row.hi && node >> 6 < p.mask_words && (row.bits[node >> 6] >> (node & 63) & 1);
    } else {
        return k >= row.lo && k < row.hi;
    }
}

// Rows of codes and scales, and the 16-byte chunks of a row.
template <int F, int D>
struct AttnGeom {
    static constexpr int RB = F == FMT_FP4 ? D / 2 : D;     // bytes of a key's codes
    static constexpr int SB = D / 32;                       // and of its scales
    static constexpr int CH = RB / 16;                      // chunks of a key
    static constexpr int VC = F == FMT_FP4 ? 32 : 16;       // values of a chunk
    static constexpr int NP = VC / 8;                       // pieces of eight
    // a key's scales as they are loaded: the type of what a loop carries to its
    // next turn (widened there; where the loop carries them widened, its end
    // waits for the loads that it has just issued, 3% of a long E2M1 context)
    typedef typename std::conditional<SB == 4, uint32_t, uint16_t>::type Scales;
};

// Page of key `key` of a sequence (its table row), or -1 past key1 or where
// the table names no page of the cache.
__device__ __forceinline__ int attn_page(const AttnArgs &p, const int *table, int key, int key1)
{
    int page = -1;
    if (key < key1)
        page = table[key >> p.page_shift];
    return (unsigned)page < (unsigned)p.pages ? page : -1;
}

// The same in two steps, the table's entry loaded ahead (that of the last key
// past key1; key1 > 0) and looked at when it is needed: a comparison right
// behind the load would wait for it.
__device__ __forceinline__ int attn_entry(const AttnArgs &p, const int *table, int key, int key1)
{
    return table[min(key, key1 - 1) >> p.page_shift];
}

__device__ __forceinline__ int attn_page_of(const AttnArgs &p, int entry, int key, int key1)
{
    return key < key1 && (unsigned)entry < (unsigned)p.pages ? entry : -1;
}

// Row of the cache (codes and scales) of key `key` on page `page`.  A key
// that is not there (page < 0) takes row 0: in bounds, and not used.
__device__ __forceinline__ long long attn_row_at(const AttnArgs &p, int page, int head, int key)
{
    const int off = key & ((1 << p.page_shift) - 1);
    return page >= 0 ? ((((long long)page * p.heads + head) << p.page_shift) + off) : 0;
}

// A chunk as BF16, in pieces of eight values.
template <int F, int NP>
__device__ __forceinline__ void attn_expand(const u4v &c, unsigned s, u4v (&w)[NP])
{
    if constexpr (F == FMT_FP4) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = mx_decode8<F>(u2v{c[i], 0u}, s);
    } else {
        w[0] = mx_decode8<F>(u2v{c[0], c[1]}, s);
        w[1] = mx_decode8<F>(u2v{c[2], c[3]}, s);
    }
}

// NaN or infinity
__device__ __forceinline__ bool bf16_special(unsigned x) { return (x & 0x7FFFu) >= 0x7F80u; }

// A chunk of values of a tile that not every row sees whole: zeros for a key
// that is not there and in the place of NaNs and infinities.  Returns whether
// there was one.
template <int NP>
__device__ __forceinline__ bool attn_clean(u4v (&w)[NP], bool ok)
{
    bool special = false;
#pragma unroll
    for (int e = 0; e < NP; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool a = bf16_special(w[e][i]), b = bf16_special(w[e][i] >> 16);
            special |= a | b;
            w[e][i] = ok ? w[e][i] & ((a ? 0u : 0xFFFFu) | (b ? 0u : 0xFFFF0000u)) : 0u;
        }
    return special && ok;
}

// Whether the values of a row of the cache may hold a NaN or an infinity: an
// E4M3 NaN code, or a scale under which the largest code (448 or 6, with BF16's
// 2^128 out of reach up to scale codes 246 and 252) is infinite, 255 included.
template <int F, int D>
__device__ __forceinline__ bool attn_may_be_special(const AttnArgs &p, long long at)
{
    using G = AttnGeom<F, D>;
    bool any = false;
#pragma unroll
    for (int b = 0; b < G::SB; ++b)
        any |= p.scales[1][at * G::SB + b] > (F == FMT_FP4 ? 252 : 246);
    if constexpr (F == FMT_FP8)
#pragma unroll
        for (int c = 0; c < G::CH; ++c) {
            const u4v w = *reinterpret_cast<const u4v *>(p.codes[1] + at * G::RB + 16 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                any |= (((w[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
        }
    return any;
}

__device__ __forceinline__ bool attn_finite(const float (&f)[8])
{
    float probe = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        probe = fmaf(f[e], 0.0f, probe);
    return probe == probe;
}

// Put the NaNs and infinities that a lane's row sees among values col .. col + 7
// of the item's keys into its sums f of these columns.  The whole wave looks
// through 64 keys at a time and takes those that may hold one in turn: once
// per item, and only where a sum is not finite or a value was replaced.
template <int F, int D, int TREE>
__device__ __forceinline__ void attn_special(const AttnArgs &p, const int *table, const AttnItem &it, const AttnRow<TREE> &row, int col,
                                             float (&f)[8])
{
    using G = AttnGeom<F, D>;
    unsigned pos = 0, neg = 0, nan = 0;
    for (int key = it.key0; key < it.key1; key += 64) {
        const int mine = key + ((int)threadIdx.x & 63), page = attn_page(p, table, mine, it.key1);
        bool may = false;
        if (page >= 0)
            may = attn_may_be_special<F, D>(p, attn_row_at(p, page, it.head, mine));
        unsigned long long left = __ballot(may);
        while (left) {
            const int i = __ffsll(left) - 1, k = key + i;
            left &= left - 1;
            const long long at = attn_row_at(p, lane_value(page, i), it.head, k);
            const bool see = attn_sees_key<TREE>(p, row, k);
            u2v c;
            if constexpr (F == FMT_FP4)
                c = u2v{*reinterpret_cast<const unsigned *>(p.codes[1] + at * G::RB + col / 2), 0u};
            else
                c = *reinterpret_cast<const u2v *>(p.codes[1] + at * G::RB + col);
            const u4v w = mx_decode8<F>(c, p.scales[1][at * G::SB + col / 32]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const unsigned x = w[e >> 1] >> (16 * (e & 1)) & 0xFFFFu, bit = see ? 1u << e : 0u;
                pos |= x == 0x7F80u ? bit : 0u;
                neg |= x == 0xFF80u ? bit : 0u;
                nan |= (x & 0x7FFFu) > 0x7F80u ? bit : 0u;
            }
        }
    }
    nan |= pos & neg;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        f[e] = pos >> e & 1 ? __builtin_inff() : neg >> e & 1 ? -__builtin_inff() : f[e];
        f[e] = nan >> e & 1 ? __builtin_nanf("") : f[e];
    }
}

__device__ __forceinline__ bf16x8v as_bf16x8(u4v v) { return __builtin_bit_cast(bf16x8v, v); }

// Four keys' values at one column per lane from rows of the LDS tile (see
// the kernels for the lanes' addresses).
__device__ __forceinline__ u2v lds_read_tr(const char *at)
{
    return __builtin_bit_cast(
        u2v, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4v *)at));
}

// max over the two lanes l, l ^ 32 (l ^ 16), without LDS.
__device__ __forceinline__ float max_across_32(float v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

__device__ __forceinline__ float max_across_16(float v)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// The largest sum of a lane's p of one tile that keeps the row's reference.
constexpr float kMostSum = 4096.0f;

// Eight consecutive outputs of a row, d .. d + 7.
__device__ __forceinline__ void attn_store8(const AttnArgs &p, size_t row, int dim, int d, const float (&f)[8])
{
    const size_t at = row * dim + d;
    if (p.out_kind == OUT_F32) {
        v4f *o = reinterpret_cast<v4f *>(reinterpret_cast<float *>(p.out) + at);
        o[0] = v4f{f[0], f[1], f[2], f[3]};
        o[1] = v4f{f[4], f[5], f[6], f[7]};
    } else {
        u4v *o = reinterpret_cast<u4v *>(reinterpret_cast<uint16_t *>(p.out) + at);
        if (p.out_kind == OUT_BF16)
            *o = u4v{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
        else
            *o = u4v{pack_f16(f[0], f[1]), pack_f16(f[2], f[3]), pack_f16(f[4], f[5]), pack_f16(f[6], f[7])};
    }
}

// Bytes of the workspace slot of a part of a tile of `rows` rows: the sums
// [rows][dim], then (m, l) of each row; a multiple of 128.
constexpr int attn_slot_bytes(int rows, int dim) { return rows * dim * 4 + cdiv_c(rows * 8, 128) * 128; }

// Eight sums of a row relative to m, and the sum of its p.
struct AttnSums {
    float f[8], m, l;
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = 0.0f;
        m = -__builtin_inff();
        l = 0.0f;
    }
    // (sums of keys that the row does not see: m = -inf, l = 0, f = 0.  The
    // weights stay above 0, where an infinite sum would become NaN)
    __device__ __forceinline__ void add(const float (&g)[8], float mq, float lq)
    {
        const float mn = fmaxf(m, mq);
        const float wa = m == mn ? 1.0f : fmaxf(__builtin_amdgcn_exp2f(m - mn), 0x1p-149f);
        const float wb = mq == mn ? 1.0f : fmaxf(__builtin_amdgcn_exp2f(mq - mn), 0x1p-149f);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = f[e] * wa + g[e] * wb;
        l = l * wa + lq * wb;
        m = mn;
    }
};

// Run i of a row tile (columns 8 (i % (D / 8)) .. + 7 of row i / (D / 8)):
// outputs and lse.
template <int D>
__device__ __forceinline__ void attn_write(const AttnArgs &p, const AttnItem &it, int i, AttnSums &s)
{
    constexpr int RUNS = D / 8;
    const int run = i % RUNS;
    const AttnRow<0> r = attn_row<0>(p, it, it.row0 + i / RUNS);
    const size_t row = (size_t)(it.tok0 + r.token) * (p.heads * p.group) + it.head * p.group + r.head;
    // (a row that sees no key has l = 0 and sums 0; a NaN is not 0)
    const float inv = s.l == 0.0f ? 0.0f : 1.0f / s.l;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        s.f[e] *= inv;
    attn_store8(p, row, D, 8 * run, s.f);
    if (p.lse && run == 0)
        p.lse[row] = s.l == 0.0f ? -__builtin_inff() : (s.m + __builtin_amdgcn_logf(s.l)) * 0.6931471805599453f;
}

constexpr int kDeviceScope = 16;    // cache policy of a device-scope access

// The workspace slot of a part.
template <int D, int NR>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t attn_slot(const AttnArgs &p, const AttnItem &it, int part)
{
    constexpr int SLOT = attn_slot_bytes(NR, D);
    return make_rsrc(p.parts + (size_t)(it.slot + part * it.slot_step) * SLOT, (unsigned)SLOT);
}

// Run i of this part into its slot.
template <int D, int NR>
__device__ __forceinline__ void attn_put_part(__amdgpu_buffer_rsrc_t slot, int i, const AttnSums &s)
{
    constexpr int RUNS = D / 8, SUMS = NR * D * 4;
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4v, v4f{s.f[0], s.f[1], s.f[2], s.f[3]}), slot,
                                           (unsigned)(i * 32), 0, kDeviceScope);
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4v, v4f{s.f[4], s.f[5], s.f[6], s.f[7]}), slot,
                                           (unsigned)(i * 32 + 16), 0, kDeviceScope);
    if (i % RUNS == 0)
        __builtin_amdgcn_raw_buffer_store_b64(u2v{__float_as_uint(s.m), __float_as_uint(s.l)}, slot,
                                              (unsigned)(SUMS + i / RUNS * 8), 0, kDeviceScope);
}

// Parts first, first + step, .. below `end` of run i, in that order.
template <int D, int NR>
__device__ __forceinline__ void attn_sum_parts(const AttnArgs &p, const AttnItem &it, int i, int first, int step, int end, AttnSums &s)
{
    constexpr int RUNS = D / 8, SUMS = NR * D * 4;
    s.clear();
    constexpr int PF = 8;       // parts in flight
    for (int q0 = first; q0 < end; q0 += PF * step) {
        u4v a[PF], b[PF];
        u2v ml[PF];
#pragma unroll
        for (int q = 0; q < PF; ++q) {
            const __amdgpu_buffer_rsrc_t src = attn_slot<D, NR>(p, it, min(q0 + q * step, end - 1));
            ml[q] = __builtin_amdgcn_raw_buffer_load_b64(src, (unsigned)(SUMS + i / RUNS * 8), 0, kDeviceScope);
            a[q] = __builtin_amdgcn_raw_buffer_load_b128(src, (unsigned)(i * 32), 0, kDeviceScope);
            b[q] = __builtin_amdgcn_raw_buffer_load_b128(src, (unsigned)(i * 32 + 16), 0, kDeviceScope);
        }
#pragma unroll
        for (int q = 0; q < PF; ++q)
            if (q0 + q * step < end) {
                const v4f fa = __builtin_bit_cast(v4f, a[q]), fb = __builtin_bit_cast(v4f, b[q]);
                s.add({fa[0], fa[1], fa[2], fa[3], fb[0], fb[1], fb[2], fb[3]}, __uint_as_float(ml[q][0]),
                      __uint_as_float(ml[q][1]));
            }
    }
}

// Parts first, first + step, .. below `end` of a row tile's n runs, by a
// workgroup, each run's sums to put(run, sums).  Where the runs leave threads
// over, two or four groups of threads take every second or fourth part each and
// are joined in `scratch` (40 NTHR bytes of LDS).
template <int D, int NR, int NTHR, class Put>
__device__ __forceinline__ void attn_sum_runs(const AttnArgs &p, const AttnItem &it, int tid, int n, int first, int step, int end,
                                              float *scratch, Put &&put)
{
    const int groups = n <= NTHR / 4 ? 4 : n <= NTHR / 2 ? 2 : 1;
    if (groups > 1) {
        // (whole waves per group: the first part is a scalar)
        const int each = NTHR / groups, group = uniform(tid / each), i = tid - group * each;
        AttnSums s;
        if (i < n) {
            attn_sum_parts<D, NR>(p, it, i, first + group * step, step * groups, end, s);
            if (group > 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    scratch[e * NTHR + tid] = s.f[e];
                scratch[8 * NTHR + tid] = s.m;
                scratch[9 * NTHR + tid] = s.l;
            }
        }
        __syncthreads();
        if (group == 0 && i < n) {
            for (int o = 1; o < groups; ++o) {
                const float *src = scratch + o * each + i;
                s.add({src[0], src[NTHR], src[2 * NTHR], src[3 * NTHR], src[4 * NTHR], src[5 * NTHR], src[6 * NTHR], src[7 * NTHR]},
                      src[8 * NTHR], src[9 * NTHR]);
            }
            put(i, s);
        }
    } else {
#pragma unroll 1
        for (int i = tid; i < n; i += NTHR) {
            AttnSums s;
            attn_sum_parts<D, NR>(p, it, i, first, step, end, s);
            put(i, s);
        }
    }
}

// Trees: the join of a row tile's parts, n runs of it, once this workgroup's
// are in its slot: by the workgroup that arrives last.  More than 2 kJoin
// parts are joined in two steps, kJoin of them by the last of each kJoin and
// what these leave by the last of all (one sequence of 4 nodes over 16000 keys,
// 63 parts for each of 8 heads: 29.7 us by one alone, 17.5 in two steps).
constexpr int kJoin = 8;
constexpr int kTreeTiles = 8192;        // row tiles that may be split, and as many slots

template <int D, int NR, int NTHR>
__device__ __forceinline__ void attn_join_tree(const AttnArgs &p, const AttnItem &it, int tid, int n, float *scratch)
{
    __shared__ unsigned arrived;
    auto last = [&](int counter, int of) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (tid == 0) {
            arrived = __hip_atomic_fetch_add(p.counters + counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (arrived == (unsigned)(of - 1))
                __hip_atomic_store(p.counters + counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        return arrived == (unsigned)(of - 1);
    };
    // parts first, first + step, .. below end, to the outputs or to part `to`
    auto sum = [&](int first, int step, int end, int to) {
        attn_sum_runs<D, NR, NTHR>(p, it, tid, n, first, step, end, scratch, [&](int i, AttnSums &s) {
            if (to < 0)
                attn_write<D>(p, it, i, s);
            else
                attn_put_part<D, NR>(attn_slot<D, NR>(p, it, to), i, s);
        });
    };
    if (it.parts <= 2 * kJoin) {
        if (last(it.counter, it.parts))
            sum(0, 1, it.parts, -1);
        return;
    }
    const int from = it.part / kJoin * kJoin, upto = min(from + kJoin, it.parts);
    if (upto > from + 1) {
        // (the counters behind the row tiles', by the slot of the first of them)
        if (!last(kTreeTiles + it.slot + from * it.slot_step, upto - from))
            return;
        sum(from, 1, upto, from);
    }
    if (last(it.counter, (it.parts + kJoin - 1) / kJoin))
        sum(0, kJoin, it.parts, -1);
}

// The end of a part of a row tile of few rows, of which run u of thread `tid`
// (i = tid + u NTHR, for the rows that are there) has the sums get(u, sums):
// the outputs, or where the row tile is split the part, and the whole in the
// workgroup that arrives last.
//
// That workgroup reads the parts alone, one memory latency after the other,
// which for one sequence's few rows cost more than the keys (4 rows of 64
// parts 30 of 64 us): so parts hold only the rows that are there, and several
// groups of threads share them (attn_sum_runs; `scratch`: LDS that nothing else
// uses any more).
template <int D, int NR, int NTHR, int TREE, class Get>
__device__ __forceinline__ void attn_finish(const AttnArgs &p, const AttnItem &it, int tid, float *scratch, Get &&get)
{
    constexpr int RUNS = D / 8, NU = cdiv_c(NR * RUNS, NTHR);
    const int n = min(NR, it.ntok * p.group - it.row0) * RUNS;
    const __amdgpu_buffer_rsrc_t slot = attn_slot<D, NR>(p, it, it.part);
#pragma unroll
    for (int u = 0; u < NU; ++u)
        if (tid + u * NTHR < n) {
            AttnSums s;
            get(u, s);
            if (it.parts == 1)
                attn_write<D>(p, it, tid + u * NTHR, s);
            else
                attn_put_part<D, NR>(slot, tid + u * NTHR, s);
        }
    if (it.parts == 1)
        return;
    if constexpr (TREE) {
        attn_join_tree<D, NR, NTHR>(p, it, tid, n, scratch);
        return;
    }
    __shared__ unsigned arrived;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid == 0)
        arrived = __hip_atomic_fetch_add(p.counters + it.counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (arrived != (unsigned)(it.parts - 1))
        return;
    attn_sum_runs<D, NR, NTHR>(p, it, tid, n, 0, 1, it.parts, scratch, [&](int i, AttnSums &s) { attn_write<D>(p, it, i, s); });
    if (tid == 0)
        __hip_atomic_store(p.counters + it.counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Key tiles worth a part of their own in mx_attn_tile (64 rows over 8000 keys:
// 2 tiles 34 us, 4 27, 8 25; 512 rows over 1500 keys: 8 tiles 32 us, 12 38,
// 24 50).
constexpr int kTileParts = 8;

// The join of row tiles of many rows, a kernel of its own behind mx_attn_tile:
// 512 runs of a row tile per workgroup, 256 of trees.  (The last workgroup of a
// row tile, joining alone as above, took 30 us for 31 parts of 64 rows.)
constexpr int attn_join_blocks(int rows, int dim, int tree) { return cdiv_c(rows * dim / 8, tree ? 256 : 512); }

template <int D, int BM, int TREE>
__global__ __launch_bounds__(256)
void mx_attn_join(AttnArgs p)
{
    constexpr int RUNS = D / 8, SUB = attn_join_blocks(BM, D, TREE), EACH = TREE ? 1 : 2;
    AttnItem it;
    if (!plan_item<TREE, BM, 64, 1>(p, blockIdx.x / SUB, kTileParts, it) || it.parts == 1)
        return;
    const int n = min(BM, it.ntok * p.group - it.row0) * RUNS;
#pragma unroll 1
    for (int u = 0; u < EACH; ++u) {
        const int i = (blockIdx.x % SUB * EACH + u) * 256 + threadIdx.x;
        if (i < n) {
            AttnSums s;
            attn_sum_parts<D, BM>(p, it, i, 0, 1, it.parts, s);
            attn_write<D>(p, it, i, s);
        }
    }
}

// ------------------------------------------------------------ few rows
// Row tiles of 16 QT rows.  The four waves of a workgroup take turns at tiles
// of 32 keys, each with its own sums, its own LDS and no barrier in the loop;
// the sums are joined at the end.  Bound: HBM, the cache's bytes, and close
// behind it (for MXFP4 codes before it) the VALU work of expanding them; the
// next tile's codes are in flight while one is worked on.  64 sequences of 100
// to 16000 keys, 8 KV heads of 128, E4M3: 436 MB in 93 us, 4.7 TB/s (a second
// tile in flight 100 us: its registers cost a wave); three of 60000 to 131072
// in E2M1: 349 MB in 69 us, 5.1 TB/s; one of 1025 keys 9.8 us: the launch, the
// plan, a few dependent loads and the join.
//
// v_mfma_f32_16x16x32_bf16, lane (r = l & 15, g = l >> 4): operands row r,
// k = 8g .. 8g + 7; accumulator column r, rows 4g .. 4g + 3.  So S^T tile kt
// (keys 16 kt ..) leaves lane (r, g) with keys 16 kt + 4g + i of query row r,
// and P^T's eight k of lane group g are keys 4g + i and 16 + 4g + i.
//
// Keys go from memory to the MFMA without LDS: lane (r, g) loads the g-th
// quarter of key r's row (for 128 bytes, 16 bytes of each half), and step s
// of the product takes eight values of that piece, d = column(s, g) .. + 7;
// q is loaded in the same order of d.  (16 rows in consecutive lanes cost the
// address unit three times a contiguous load, which is still twice what HBM
// delivers; through LDS the keys took 8 writes, 8 reads and a round trip per
// tile.)
//
// Values are expanded into LDS as rows of 2D + 32 bytes and read transposed
// (the 32 spread the four keys and four lane groups of a read over the banks).
//
// PAGED: pages of 16 keys or more, so that the two pages of a tile are
// scalars and the lanes' offsets the same for every tile.
template <int F, int D, int QT, int PAGED, int TREE, int P2>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(QT > 1 ? 2 : F == FMT_FP8 && D == 128 ? 3 : 4)))
void mx_attn_rows(AttnArgs p)
{
    constexpr int KT = 32, BM = 16 * QT, BN = 4 * KT;
    using G = AttnGeom<F, D>;
    constexpr int KS = D / 32, DT = D / 16, NP = G::NP;
    constexpr int KPL = 64 / G::CH, NL = KT / KPL;      // values: keys per load, loads per tile
    constexpr int KQ = G::RB / 4;                       // bytes of a key's row per lane: 8, 16 or 2 x 16
    constexpr int VROW = 2 * D + 32, WBYTES = KT * VROW;
    constexpr int OROW = D + 4;                         // floats of a row of sums in LDS
    constexpr int OBYTES = 16 * OROW * 4;               // one wave's 16 rows
    constexpr int BYTES = (WBYTES > OBYTES ? WBYTES : OBYTES) * 4;
    __shared__ __attribute__((aligned(1024))) char lds[BYTES];
    __shared__ float ml[4][BM][2];
    __shared__ unsigned cleaned[4];                     // a wave replaced a value by a zero
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), r = lane & 15, g = lane >> 4;

    AttnItem it;
    if (!plan_item<TREE, BM, BN>(p, blockIdx.x, 2, it))
        return;

    const int *table = p.table + it.seq * p.table_stride;
    int key = it.key0 + wave * KT;
    // table entry of key `lane & 31` of the next tile loaded
    int entry = it.key0 < it.key1 ? attn_entry(p, table, key + (lane & 31), it.key1) : -1;

    // first of the eight columns that step s takes from this lane
    auto column = [&](int s) {
        return F == FMT_FP4 ? (D / 4) * g + 8 * s : D == 128 ? (s >> 1) * 64 + 16 * g + 8 * (s & 1) : (D / 4) * g + 8 * s;
    };
    AttnRow<TREE> row[QT];
    bf16x8v q[QT][KS];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        row[t] = attn_row<TREE>(p, it, it.row0 + 16 * t + r);
        const uint16_t *src = p.q + (long long)(it.tok0 + max(row[t].token, 0)) * p.q_stride +
                              (long long)(it.head * p.group + row[t].head) * D;
#pragma unroll
        for (int s = 0; s < KS; ++s)
            q[t][s] = as_bf16x8(row[t].token >= 0 ? *reinterpret_cast<const u4v *>(src + column(s)) : u4v{0u, 0u, 0u, 0u});
    }

    char *mem = lds + wave * WBYTES;
    v4f o[QT][DT];
    float m[QT], l[QT];
    bool replaced = false;          // a value, by a zero
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        // (0 for rows that are not there, whose scores are 0)
        m[t] = row[t].token >= 0 ? -__builtin_inff() : 0.0f;
        l[t] = 0.0f;
#pragma unroll
        for (int d = 0; d < DT; ++d)
            o[t][d] = v4f{0, 0, 0, 0};
    }

    // The next tile: this lane's pieces of keys r and 16 + r with the row's
    // scale codes, its chunks of values (key mykey + j KPL) with theirs, and
    // the keys of it that are there (bits).
    u4v kc[2][2], vc[NL];
    typename G::Scales ks[2];
    uint8_t vs[NL];
    unsigned there = 0;
    const int mykey = lane / G::CH, chunk = lane % G::CH;
    auto load = [&](int k) {
        const int page = attn_page_of(p, entry, k + (lane & 31), it.key1);
        there = (unsigned)__ballot(page >= 0);
        // rows of the cache of keys 0 and 16 of the tile
        long long at0 = 0, at1 = 0;
        if constexpr (PAGED) {
            at0 = attn_row_at(p, lane_value(page, 0), it.head, k);
            at1 = attn_row_at(p, lane_value(page, 16), it.head, k + 16);
        }
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
            long long at = kt ? at1 : at0;
            unsigned off = r;                           // rows on from there
            if constexpr (!PAGED) {
                at = attn_row_at(p, __shfl(page, 16 * kt + r), it.head, k + 16 * kt + r);
                off = 0;
            }
            const uint8_t *c = p.codes[0] + at * G::RB, *s = p.scales[0] + at * G::SB;
            if constexpr (KQ == 8) {
                const u2v w = *reinterpret_cast<const u2v *>(c + (off * G::RB + 8 * g));
                kc[kt][0] = u4v{w.x, w.y, 0u, 0u};
            } else {
                kc[kt][0] = *reinterpret_cast<const u4v *>(c + (off * G::RB + 16 * g));
                if constexpr (KQ == 32)
                    kc[kt][1] = *reinterpret_cast<const u4v *>(c + (off * G::RB + 64 + 16 * g));
            }
            ks[kt] = *reinterpret_cast<const typename G::Scales *>(s + off * G::SB);
        }
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            const int kk = mykey + j * KPL;
            long long at;
            unsigned off;
            if constexpr (!PAGED) {
                at = attn_row_at(p, __shfl(page, kk), it.head, k + kk);
                off = 0;
            } else if constexpr (KPL <= 16) {
                at = j * KPL < 16 ? at0 : at1;
                off = kk & 15;
            } else {
                at = kk < 16 ? at0 : at1;
                off = kk & 15;
            }
            vc[j] = *reinterpret_cast<const u4v *>(p.codes[1] + at * G::RB + (off * G::RB + 16 * chunk));
            vs[j] = (p.scales[1] + at * G::SB)[off * G::SB + chunk * G::VC / 32];
        }
        entry = attn_entry(p, table, k + BN + (lane & 31), it.key1);
    };
    auto wave_fence = [] {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    };
    if (key < it.key1)
        load(key);
    char *vput = mem + mykey * VROW + chunk * G::VC * 2;
    const char *vread = mem + (4 * g + (r >> 2)) * VROW + (r & 3) * 8;
    for (; key < it.key1; key += BN) {
        // values into LDS
        const bool whole = there == 0xFFFFFFFFu && key >= it.all_lo && key + KT <= it.all_hi;
        const unsigned here = there;
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            u4v w[NP];
            attn_expand<F>(vc[j], vs[j], w);
            if (__builtin_expect(!whole, 0))
                replaced |= attn_clean(w, here >> (mykey + j * KPL) & 1);
#pragma unroll
            for (int e = 0; e < NP; ++e)
                *reinterpret_cast<u4v *>(vput + j * KPL * VROW + 16 * e) = w[e];
        }
        // scores: step s takes piece s & 1 (of an E4M3 chunk) or s & 3
        v4f x[QT][2];
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                u4v w;
                if constexpr (F == FMT_FP4) {
                    const unsigned byte = D == 128 ? ks[kt] >> (8 * g) & 255u : ks[kt] >> (8 * (g >> 1)) & 255u;
                    w = mx_decode8<F>(u2v{kc[kt][0][s], 0u}, byte);
                } else {
                    const unsigned byte = ks[kt] >> (8 * (g >> 1) + (D == 128 ? 16 * (s >> 1) : 0)) & 255u;
                    w = mx_decode8<F>(u2v{kc[kt][s >> 1][2 * (s & 1)], kc[kt][s >> 1][2 * (s & 1) + 1]}, byte);
                }
#pragma unroll
                for (int t = 0; t < QT; ++t)
                    x[t][kt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(w), q[t][s], s ? x[t][kt] : v4f{0, 0, 0, 0}, 0, 0, 0);
            }
        // (past the last key: row 0 of the cache, not used.  Under a condition
        // the loop would wait for the loads it has just issued, to merge them
        // with the registers' old contents)
        load(key + BN);
        bf16x8v pb[QT], rest[P2 ? QT : 1];
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            if (!whole) {
                const unsigned see = (unsigned)attn_sees<TREE>(p, row[t], key) & here;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[t][e >> 2][e & 3] = see >> (4 * g) >> (16 * (e >> 2) + (e & 3)) & 1 ? x[t][e >> 2][e & 3] : -__builtin_inff();
            }
            auto weights = [&](float ref) {
                float sum = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float w = __builtin_amdgcn_exp2f(fmaf(x[t][e >> 2][e & 3], p.c, -ref));
                    sum += w;
                    pb[t][e] = (__bf16)w;
                    if constexpr (P2)
                        rest[t][e] = (__bf16)(w - (float)pb[t][e]);
                }
                return sum;
            };
            float sum = 0.0f;
            bool raise = key < it.key0 + BN;        // the wave's first tile
            if (!raise) {
                sum = weights(m[t]);
                raise = __any(!(sum <= kMostSum));
            }
            if (__builtin_expect(raise, 0)) {
                float top = -__builtin_inff();
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    top = fmaxf(top, x[t][e >> 2][e & 3]);
                const float mn = fmaxf(m[t], max_across_32(max_across_16(top)) * p.c);
                const float w = m[t] == mn ? 1.0f : __builtin_amdgcn_exp2f(m[t] - mn);
                l[t] *= w;
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        o[t][d][i] *= w;
                m[t] = mn;
                // (no key seen yet: m = -inf, every x = -inf, p = 0)
                sum = weights(mn == -__builtin_inff() ? 0.0f : mn);
            }
            l[t] += sum;
        }
        wave_fence();
        // values of keys 4g .. and 16 + 4g .., columns 16 d + r
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            const u2v a = lds_read_tr(vread + 32 * d), b = lds_read_tr(vread + 16 * VROW + 32 * d);
            const bf16x8v f = as_bf16x8(u4v{a.x, a.y, b.x, b.y});
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                o[t][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, pb[t], o[t][d], 0, 0, 0);
                if constexpr (P2)
                    o[t][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, rest[t], o[t][d], 0, 0, 0);
            }
        }
        wave_fence();
    }

    // join the four waves, 16 rows at a time
    replaced = __any(replaced);
    if (lane == 0)
        cleaned[wave] = replaced;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        l[t] += __shfl_xor(l[t], 16);
        l[t] += __shfl_xor(l[t], 32);
        if (g == 0) {
            ml[wave][16 * t + r][0] = m[t];
            ml[wave][16 * t + r][1] = l[t];
        }
    }
    __syncthreads();
    // (run i of the 16 QT rows' runs of eight columns: thread i % 256)
    constexpr int RUNS = D / 8, NU = cdiv_c(BM * RUNS, 256);
    float f[NU][8], fm[NU], fl[NU];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        float top = -__builtin_inff();
#pragma unroll
        for (int w = 0; w < 4; ++w)
            top = fmaxf(top, ml[w][16 * t + r][0]);
        const float w = m[t] == top ? 1.0f : __builtin_amdgcn_exp2f(m[t] - top);
        float *mine = reinterpret_cast<float *>(lds) + wave * (OBYTES / 4) + r * OROW + 4 * g;
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            v4f s = o[t][d];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                s[i] *= w;
            *reinterpret_cast<v4f *>(mine + 16 * d) = s;
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            if (256 * (u + 1) <= t * 16 * RUNS || 256 * u >= (t + 1) * 16 * RUNS)
                continue;
            const int i = tid + 256 * u, n = i / RUNS, col = i % RUNS * 8;
            if (n >> 4 != t)
                continue;
            fm[u] = -__builtin_inff();
            fl[u] = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[u][e] = 0.0f;
#pragma unroll
            for (int v = 0; v < 4; ++v)
                fm[u] = fmaxf(fm[u], ml[v][n][0]);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const float mv = ml[v][n][0];
                fl[u] += ml[v][n][1] * (mv == fm[u] ? 1.0f : __builtin_amdgcn_exp2f(mv - fm[u]));
                const float *src = reinterpret_cast<const float *>(lds) + v * (OBYTES / 4) + (n & 15) * OROW + col;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[u][e] += src[e];
            }
        }
        __syncthreads();
    }
    const bool cleans = cleaned[0] | cleaned[1] | cleaned[2] | cleaned[3];
#pragma unroll
    for (int u = 0; u < NU; ++u) {
        const int i = tid + 256 * u;
        if (i - lane >= BM * RUNS)
            continue;
        const AttnRow<TREE> at = attn_row<TREE>(p, it, it.row0 + i / RUNS);
        // (a row with a NaN among its scores has l = NaN and becomes NaN)
        if (__builtin_expect(__any(at.token >= 0 && fl[u] == fl[u] && (cleans || !attn_finite(f[u]))), 0))
            attn_special<F, D, TREE>(p, table, it, at, i % RUNS * 8, f[u]);
    }
    static_assert(BYTES >= 40 * 256, "scratch");
    attn_finish<D, BM, 256, TREE>(p, it, tid, reinterpret_cast<float *>(lds), [&](int u, AttnSums &out) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            out.f[e] = f[u][e];
        out.m = fm[u];
        out.l = fl[u];
    });
}

// ------------------------------------------------------------ many rows
// Slot permutation of a key's row of values in LDS: slot p (16 bytes) of the
// row lies at p ^ value_swizzle.  A row of 128 values is the 256 bytes of all
// banks, one of 64 values half of them.
template <int D>
__device__ __forceinline__ int value_swizzle(int key)
{
    return D >= 128 ? (key & 3) * 5 : (key >> 1 & 1) * 4 + (key >> 1 & 3);
}

// Row tiles of 32 NW rows, 32 per wave, over tiles of 64 keys that the waves
// expand together.  A wave alternates between two phases:
//     M(t)   the second product of tile t - 1 and the first of tile t: MFMA,
//            fed from LDS, and between them expanding tile t + 1's codes
//            into LDS and the loads of tile t + 2's
//     V(t)   the softmax of tile t: VALU
// Bound: MFMA, and beside it VALU issue: 4096 tokens of 32 heads of 128 over
// 8 KV heads behind 12204 keys in E4M3 (0.96 TFLOP) take 820 to 861 us, 1.1
// PFLOP/s; their MFMAs alone 526 us, with the LDS reads 575, with the softmax 785.
//
// With NW = 8 the two waves of a SIMD are of different groups (waves 0-3 and
// 4-7): the one barrier per tile stands behind V for the first and behind M
// for the second, so one's M runs beside the other's V.  Between barriers t -
// 1 and t both groups are at M(t): they read keys t and values t - 1 and write
// tile t + 1, so two buffers of keys and three of values keep them apart.
// With NW = 4 (fewer rows to waste, two workgroups per CU): a barrier behind
// each phase, the expansion and the loads in V, one buffer of keys and two of
// values.
//
// v_mfma_f32_32x32x16_bf16, lane (r = l & 31, h = l >> 5): operands row r,
// k = 8h .. 8h + 7; accumulator column r, register i row 8 (i >> 2) + 4h +
// (i & 3).  So P^T's eight k of step s and half h are keys 16s + 4h + i and
// 16s + 8 + 4h + i of the tile.
//
// LDS of a buffer: the keys as operand fragments (lane order, 1 KB each,
// apart by 1 KB + 4096 / D bytes), or the values as rows of 2D bytes whose
// 16-byte slots are permuted by the key (value_swizzle).  Both so that 16
// lanes of an expanding store (the chunks of a few keys) and 32 lanes of a
// transposing read (four keys, 64 bytes of each) touch every bank once: with
// rows and fragments padded by 64 and 128 bytes the LDS spent 1000 of 2400
// busy cycles per tile on conflicts.
//
// PAGED as in mx_attn_rows.
// Tiles of 64 keys from a key on: [first, first + n).
struct TileRange {
    int first, n;
    __device__ __forceinline__ bool has(int t) const { return (unsigned)(t - first) < (unsigned)n; }
};

// those within keys [lo, hi), and those that hold one of them
__device__ __forceinline__ TileRange tiles_within(int key0, int lo, int hi)
{
    const int a = (max(lo - key0, 0) + 63) / 64, b = hi > key0 ? (hi - key0) / 64 : 0;
    return {a, max(b - a, 0)};
}

__device__ __forceinline__ TileRange tiles_touching(int key0, int lo, int hi)
{
    const int a = max(lo - key0, 0) / 64, b = hi > key0 ? (hi - key0 + 63) / 64 : 0;
    return {a, lo < hi ? max(b - a, 0) : 0};
}

template <int F, int D, int NW, int PAGED, int TREE, int P2>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(2, 2)))
void mx_attn_tile(AttnArgs p)
{
    constexpr int BM = 32 * NW, BN = 64, THR = 64 * NW;
    using G = AttnGeom<F, D>;
    constexpr int KS = D / 16, DT = D / 32, NP = G::NP;
    constexpr int KBUFS = NW == 8 ? 2 : 1, VBUFS = NW == 8 ? 3 : 2;
    constexpr int FS = 1024 + 4096 / D, KBYTES = 2 * KS * FS, VROW = 2 * D, VBYTES = BN * VROW;
    constexpr int OROW = D + 4;
    constexpr int TILES = KBUFS * KBYTES + VBUFS * VBYTES;
    constexpr int BYTES = TILES > BM * OROW * 4 ? TILES : BM * OROW * 4;
    // chunk n of the 2 x 64 CH of a tile (keys, then values): thread n % THR.
    // A wave's chunks are of one side (with SIDE >= THR known at compile time)
    // and of KPW consecutive keys from wave * KPW + i * THR / CH on.
    constexpr int SIDE = BN * G::CH, NI = cdiv_c(2 * SIDE, THR), KPW = 64 / G::CH;
    constexpr bool EVERY = 2 * SIDE >= THR, STATIC = SIDE >= THR;
    __shared__ __attribute__((aligned(1024))) char lds[BYTES];
    __shared__ float ml[BM][2];
    __shared__ unsigned cleaned[NW];                    // a wave replaced a value by a zero
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), r = lane & 31, h = lane >> 5;

    AttnItem it;
    if (!plan_item<TREE, BM, BN>(p, blockIdx.x, kTileParts, it))
        return;

    const int *table = p.table + it.seq * p.table_stride;
    const int T = (it.key1 - it.key0 + BN - 1) / BN;
    // table entry of key `lane` of the next tile loaded
    int entry = T > 0 ? attn_entry(p, table, it.key0 + lane, it.key1) : -1;
    const int chunk = tid % G::CH;                                  // THR is a multiple of CH

    const AttnRow<TREE> row = attn_row<TREE>(p, it, it.row0 + 32 * wave + r);
    bf16x8v q[KS];
    {
        const uint16_t *src = p.q + (long long)(it.tok0 + max(row.token, 0)) * p.q_stride +
                              (long long)(it.head * p.group + row.head) * D + 8 * h;
#pragma unroll
        for (int s = 0; s < KS; ++s)
            q[s] = as_bf16x8(row.token >= 0 ? *reinterpret_cast<const u4v *>(src + 16 * s) : u4v{0u, 0u, 0u, 0u});
    }
    // tiles whose keys every row of the wave sees (of those that are there),
    // and tiles of which some row may see some
    int lo_most = row.token >= 0 ? row.lo : 0, hi_least = row.token >= 0 ? (TREE ? it.all_hi : row.hi) : 0x7FFFFFFF;
    int lo_least = row.token >= 0 ? row.lo : 0x7FFFFFFF, hi_most = row.hi;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        lo_most = max(lo_most, __shfl_xor(lo_most, d));
        hi_least = min(hi_least, __shfl_xor(hi_least, d));
        lo_least = min(lo_least, __shfl_xor(lo_least, d));
        hi_most = max(hi_most, __shfl_xor(hi_most, d));
    }
    const TileRange full = tiles_within(it.key0, uniform(lo_most), uniform(hi_least));
    const TileRange some = tiles_touching(it.key0, uniform(lo_least), uniform(min(hi_most, it.key1)));
    const TileRange all_full = tiles_within(it.key0, it.all_lo, it.all_hi);     // of the whole row tile
    int gone = -1;                          // the last tile expanded so far with keys that are not there

    v16f o[DT], x[2];
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            o[d][i] = 0.0f;
    // (0 for rows that are not there, whose scores are 0)
    float m = row.token >= 0 ? -__builtin_inff() : 0.0f, l = 0.0f;
    bf16x8v pb[4], rest[P2 ? 4 : 1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        pb[i] = as_bf16x8(u4v{0u, 0u, 0u, 0u});
        if constexpr (P2)
            rest[i] = pb[i];
    }

    // the loaded tile: this thread's chunks, and the keys that are there
    u4v codes[NI];
    unsigned scale[NI];
    unsigned long long loaded = 0;
    // (threads without a chunk load an earlier one's and do not expand it)
    const bool loads = EVERY || tid < 2 * SIDE;
    const int myside = STATIC ? 0 : uniform(wave * 64 / SIDE);
    auto side_of = [&](int i) { return STATIC ? i * THR / SIDE : myside & 1; };
    auto key_of = [&](int i) { return STATIC ? wave * KPW + i * THR % SIDE / G::CH : (wave * KPW) & (BN - 1); };
    const int mykey = lane / G::CH;
    // rows of the cache per page, and of the pages before this head's
    const int page_rows = p.heads << p.page_shift, head_row = it.head << p.page_shift, in_page = (1 << p.page_shift) - 1;
    const unsigned voff = mykey * G::RB + 16 * chunk, soff = mykey * G::SB + chunk * G::VC / 32;
    // loading tile t: which keys are there, chunk i, the next tile's entries
    int page = -1;
    auto load_pages = [&](int t) {
        page = attn_page_of(p, entry, it.key0 + t * BN + lane, it.key1);
        loaded = __ballot(page >= 0);
    };
    // (for a page of the cache the row of the wave's first key is a scalar; a
    // key that is not there: of page 0, in bounds and not used)
    long long rows_at[NI];
    auto load_row = [&](int t, int i) {
        const int key = it.key0 + t * BN, k0 = key_of(i);
        if constexpr (PAGED)
            rows_at[i] = (long long)((unsigned long long)(unsigned)max(lane_value(page, k0), 0) * (unsigned)page_rows +
                                     (unsigned)(head_row + ((key + k0) & in_page)));
        else
            rows_at[i] = attn_row_at(p, __shfl(page, k0 + mykey), it.head, key + k0 + mykey);
    };
    auto load_codes = [&](int i) {
        const uint8_t *cp = side_of(i) ? p.codes[1] : p.codes[0];
        codes[i] = *reinterpret_cast<const u4v *>(cp + rows_at[i] * G::RB + (PAGED ? voff : 16u * chunk));
    };
    auto load_scale = [&](int i) {
        const uint8_t *sp = side_of(i) ? p.scales[1] : p.scales[0];
        scale[i] = (sp + rows_at[i] * G::SB)[PAGED ? soff : (unsigned)chunk * G::VC / 32];
    };
    auto load_entry = [&](int t) { entry = attn_entry(p, table, it.key0 + (t + 1) * BN + lane, it.key1); };
    auto load = [&](int t) {
        load_pages(t);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            load_row(t, i);
            load_codes(i);
            load_scale(i);
        }
        load_entry(t);
    };
    // where this thread's chunks go in a buffer of keys and one of values
    auto put_key = [&](int i, int e) {
        const int kk = key_of(i) + mykey, piece = chunk * NP + e;
        return ((kk >> 5) * KS + (piece >> 1)) * FS + (piece & 1) * 512 + (kk & 31) * 16;
    };
    auto put_value = [&](int i, int e) {
        const int kk = key_of(i) + mykey;
        return kk * VROW + 16 * ((chunk * NP + e) ^ value_swizzle<D>(kk));
    };
    // piece u of the loaded tile t into its buffer
    auto expand_piece = [&](int t, int u) {
        const int i = u / NP, e = u % NP;
        char *buf = side_of(i) ? lds + KBUFS * KBYTES + (unsigned)t % VBUFS * VBYTES
                               : lds + (KBUFS == 1 ? 0 : (unsigned)t % KBUFS) * KBYTES;
        const u2v c = F == FMT_FP4 ? u2v{codes[i][e], 0u} : u2v{codes[i][2 * e & 3], codes[i][(2 * e + 1) & 3]};
        if (loads)
            *reinterpret_cast<u4v *>(buf + (side_of(i) ? put_value(i, e) : put_key(i, e))) = mx_decode8<F>(c, scale[i]);
    };
    // once its pieces are there: what of its values has to be replaced
    auto expand_rest = [&](int t) {
        gone = loaded == ~0ull || t >= T ? gone : t;
        if (__builtin_expect(!(gone != t && all_full.has(t)), 0)) {
            char *vbuf = lds + KBUFS * KBYTES + (unsigned)t % VBUFS * VBYTES;
            bool replaced = false;
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if (side_of(i)) {
                    u4v w[NP];
                    attn_expand<F>(codes[i], scale[i], w);
                    replaced |= attn_clean(w, loaded >> (key_of(i) + mykey) & 1) && loads;
                    if (loads)
#pragma unroll
                        for (int e = 0; e < NP; ++e)
                            *reinterpret_cast<u4v *>(vbuf + put_value(i, e)) = w[e];
                }
            if (__any(replaced) && lane == 0)
                cleaned[wave] = 1;
        }
    };
    auto expand = [&](int t) {
#pragma unroll
        for (int u = 0; u < NI * NP; ++u)
            expand_piece(t, u);
        expand_rest(t);
    };
    // this lane's piece of a transposing read: key 4h + (r & 15) / 4 of eight,
    // 8 bytes r & 3 of the 32 at column group r >> 4 (eight keys on, and 64
    // bytes on, the permutation is the same but for the 64's own slots)
    const int vkey = 4 * h + ((r & 15) >> 2);
    const int vread = vkey * VROW + 8 * (r & 1), vslot = 2 * (r >> 4) + ((r & 3) >> 1);

    // The M phase is eight batches of DT MFMAs with their LDS reads two
    // batches ahead: 0 .. 3 the second product's steps of 16 keys of tile
    // t - 1, 4 .. 7 a quarter of the first product of tile t.
    u4v frag[3][DT];
    auto fetch = [&](auto bc, int t) {
        constexpr int b = decltype(bc)::value;
        if constexpr (b < 4) {
            // values of keys 16 b + 4h .. and 16 b + 8 + 4h .., columns 32 d + r
            const char *at = lds + KBUFS * KBYTES + (unsigned)max(t - 1, 0) % VBUFS * VBYTES + vread + 16 * b * VROW;
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const char *slot = at + 16 * ((4 * d + vslot) ^ value_swizzle<D>(vkey));
                const u2v lo = lds_read_tr(slot), hi = lds_read_tr(slot + 8 * VROW);
                frag[b % 3][d] = u4v{lo.x, lo.y, hi.x, hi.y};
            }
        } else {
            const char *at = lds + (KBUFS == 1 ? 0 : (unsigned)t % KBUFS) * KBYTES + lane * 16;
#pragma unroll
            for (int i = 0; i < DT; ++i)
                frag[b % 3][i] = *reinterpret_cast<const u4v *>(at + ((i & 1) * KS + (b - 4) * (DT / 2) + (i >> 1)) * FS);
        }
    };
    // With NW = 8 the M phase also expands tile t + 1 and loads tile t + 2, a
    // piece behind each of its first MFMAs: they issue while the MFMA runs,
    // where in the V phase they made it the longer one (V 2200 cycles to M's
    // 1400).
    auto between = [&](auto nc, int t) {
        constexpr int n = decltype(nc)::value;
        if constexpr (NW == 8) {
            if constexpr (n % 2 == 1 && n / 2 < NI * NP)
                expand_piece(t + 1, n / 2);
            if constexpr (n == 8)
                expand_rest(t + 1);
            if constexpr (n == 9)
                load_pages(t + 2);
            if constexpr (n == 10)
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    load_row(t + 2, i);
            if constexpr (n == 11)
                load_codes(0);
            if constexpr (n == 12)
                load_scale(0);
            if constexpr (n == 13 && NI > 1)
                load_codes(1);
            if constexpr (n == 14 && NI > 1)
                load_scale(1);
            if constexpr (n == 15)
                load_entry(t + 2);
        }
    };
    static_assert(NW != 8 || (NI <= 2 && NI * NP <= 4), "pieces in front of the loads");
    auto multiply = [&](auto bc, int t) {
        constexpr int b = decltype(bc)::value;
        static_range<0, DT>([&](auto ic) {
            constexpr int i = decltype(ic)::value;
            const bf16x8v f = as_bf16x8(frag[b % 3][i]);
            if constexpr (b < 4) {
                o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, pb[b], o[i], 0, 0, 0);
                if constexpr (P2)
                    o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, rest[b], o[i], 0, 0, 0);
            } else {
                constexpr int s = (b - 4) * (DT / 2) + (i >> 1);
                if constexpr (s == 0)
                    x[i & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, q[0], v16f{}, 0, 0, 0);
                else
                    x[i & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, q[s], x[i & 1], 0, 0, 0);
            }
            if constexpr (NW == 8) {
                __builtin_amdgcn_sched_barrier(0);
                between(IntC<b * DT + i>{}, t);
                __builtin_amdgcn_sched_barrier(0);
            }
        });
    };
    auto batches = [&](int t) {
        static_range<0, 8>([&](auto b) {
            constexpr int i = decltype(b)::value;
            if constexpr (i + 2 < 8)
                fetch(IntC<i + 2>{}, t);
            __builtin_amdgcn_sched_barrier(0);
            multiply(b, t);
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    // (always inlined: as a call its arrays would live in scratch memory)
    auto phase_m = [&](int t) __attribute__((always_inline)) {
        if constexpr (NW != 8)
            fetch(IntC<0>{}, t);
        fetch(IntC<1>{}, t);
        // (the MFMAs go first where both waves of a SIMD have something to issue)
        __builtin_amdgcn_s_setprio(1);
        // No branches, so that the sums stay in their registers: where a wave
        // saw nothing of tile t - 1 its p are zeros, and the values finite (a
        // tile that not every row sees whole holds no NaN and no infinity);
        // t = 0 takes tile 0's values for those before it, whose NaNs and
        // infinities every row sees, and gets from attn_special, where it
        // holds any.  Past the last tile the first product is not used.
        batches(t);
        __builtin_amdgcn_s_setprio(0);
    };
    auto softmax = [&](int t) {
        if (__builtin_expect(!(t > gone && full.has(t)), 0)) {
            const int key = it.key0 + t * BN;
            const unsigned long long there = __ballot(attn_page(p, table, key + lane, it.key1) >= 0);
            const unsigned long long see = (attn_sees<TREE>(p, row, key) & there) >> (4 * h);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                const unsigned half = e < 16 ? (unsigned)see : (unsigned)(see >> 32);
                x[e >> 4][e & 15] = half >> (8 * ((e & 15) >> 2) + (e & 3)) & 1 ? x[e >> 4][e & 15] : -__builtin_inff();
            }
        }
        // p under the reference so far; where their sum says that it is far
        // too low (or there is none yet: an infinity or NaN), a new one
        auto weights = [&](float ref) {
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                const float w = __builtin_amdgcn_exp2f(fmaf(x[e >> 4][e & 15], p.c, -ref));
                sum += w;
                pb[e >> 3][e & 7] = (__bf16)w;
                if constexpr (P2)
                    rest[e >> 3][e & 7] = (__bf16)(w - (float)pb[e >> 3][e & 7]);
            }
            return sum;
        };
        float sum = weights(m);
        if (__builtin_expect(__any(!(sum <= kMostSum)), 0)) {
            float top = -__builtin_inff();
#pragma unroll
            for (int e = 0; e < 32; ++e)
                top = fmaxf(top, x[e >> 4][e & 15]);
            const float mn = fmaxf(m, max_across_32(top) * p.c);
            const float w = m == mn ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
            l *= w;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    o[d][i] *= w;
            m = mn;
            // (no key seen yet: m = -inf, every x = -inf, p = 0)
            sum = weights(m == -__builtin_inff() ? 0.0f : m);
        }
        l += sum;
    };

    auto phase_v = [&](int t) {
        // the first reads of M(t + 1), whose values are there since the last
        // barrier: at its start all four waves would wait for them
        if constexpr (NW == 8) {
            fetch(IntC<0>{}, t + 1);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (some.has(t)) {
            softmax(t);
        } else {
            // (p of a tile that no row of the wave sees; and said for x as well,
            // so that nothing keeps its registers through the other phase)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                pb[i] = as_bf16x8(u4v{0u, 0u, 0u, 0u});
                if constexpr (P2)
                    rest[i] = pb[i];
            }
        }
        // (loads past the last tile are of page 0 of the cache and not used.
        // Under a condition the loop would wait for the loads it has just
        // issued, to merge them with the registers' old contents)
        if constexpr (NW != 8) {
            expand(t + 1);
            load(t + 2);
        }
    };
    if (lane == 0)
        cleaned[wave] = 0;
    if (T > 0) {
        load(0);
        expand(0);
        load(1);
        block_barrier();
        if constexpr (NW == 8)
            fetch(IntC<0>{}, 0);
        if (NW == 8 && wave >= 4) {
            for (int i = 0; i < T; ++i) {
                const int t = opaque(i);
                phase_m(t);
                block_barrier();
                phase_v(t);
            }
        } else {
            for (int i = 0; i < T; ++i) {
                const int t = opaque(i);
                phase_m(t);
                if (NW != 8)
                    block_barrier();
                phase_v(t);
                block_barrier();
            }
        }
        phase_m(T);
    }
    __syncthreads();
    l += __shfl_xor(l, 32);
    if (h == 0) {
        ml[32 * wave + r][0] = m;
        ml[32 * wave + r][1] = l;
    }
    float *mine = reinterpret_cast<float *>(lds) + (32 * wave + r) * OROW + 4 * h;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<v4f *>(mine + 32 * d + 8 * i) = v4f{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
    __syncthreads();
    constexpr int RUNS = D / 8;
    const int n = min(BM, it.ntok * p.group - it.row0) * RUNS;
    const __amdgpu_buffer_rsrc_t slot = attn_slot<D, BM>(p, it, it.part);
    bool cleans = false;
#pragma unroll
    for (int w = 0; w < NW; ++w)
        cleans |= cleaned[w] != 0;
    for (int i = tid; i - lane < n; i += THR) {         // (whole waves)
        const int rr = i / RUNS;
        const float *src = reinterpret_cast<const float *>(lds) + rr * OROW + i % RUNS * 8;
        AttnSums s;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            s.f[e] = src[e];
        s.m = ml[rr][0];
        s.l = ml[rr][1];
        // (a row with a NaN among its scores has l = NaN and becomes NaN)
        if (__builtin_expect(__any(i < n && s.l == s.l && (cleans || !attn_finite(s.f))), 0))
            attn_special<F, D, TREE>(p, table, it, attn_row<TREE>(p, it, it.row0 + rr), i % RUNS * 8, s.f);
        if (i >= n)
            continue;
        if (it.parts == 1)
            attn_write<D>(p, it, i, s);
        else
            attn_put_part<D, BM>(slot, i, s);
    }
}

}  // namespace mxg
