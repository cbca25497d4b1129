// attn_paged.cuh — attention of a ragged batch of new tokens over a paged cache, on
// the tensor cores: the kernels and their launch. attn_paged.cu, attn_paged_tree.cu
// and attn_paged_fp8.cu build the variants (below).
//
// Mathematics: per (sequence, key/value head) the G query heads of the group and a
// run of new tokens are packed as rows of a 128-row M tile (row = token * G + head
// in the group), so grouped heads share every key/value tile they read. A unit of
// work is NT such tiles (1 when a whole sequence's rows fit one tile, as in decode;
// 2 for prompt chunks, so that one tile's softmax overlaps the other's products)
// against the sequence's key tiles of 128. The loop over key tiles is the online
// softmax of the other forward kernels: S = Q K^T in tensor memory, P = 2^(S - m)
// rounded to the 16-bit type, O += P V, with a reference max that moves only when
// a tile's max exceeds it by more than 8 (log2 units).
//
// What bounds it: decode reads every key and value once for a few products each, so
// HBM (a ragged batch of 64 sequences of 4096-8192 keys: 238-245 us from one GPU to
// another, 6.6-6.8 TB/s, 98-101 % of the measured copy rate; 96-99 % with 16-token
// pages); long chunks by the products and their issue (4096 rows over 32768 keys: 1.26
// ms, 1635 TFLOP/s, 88 % of the GEMM rate measured in bursts, where single calls are
// timed; call after call the power cap lowers the clock, 1.41-1.46 ms, 83-86 % of the
// sustained GEMM rate. Of about 3000 cycles a key tile the products take 2050 at their
// nominal rate, an S product rather 72-87 cycles than 64 since it reads 8 KB of shared
// memory, and the issuer's turns between the two tiles the rest; the softmax of a tile
// takes 1140 and waits); small calls by latency (one token over 517 keys: 10.3 us for
// both launches, of which locating the work takes 1.4, the first copies 2, the merge 3).
//
// The calls that figures here and below name have 32 query and 8 key/value heads,
// d = 128, bf16, pages of 64 tokens, one new token a sequence and causal rows, unless
// they say otherwise. "N sequences of K keys" are ragged: lengths from 70 % of K to K
// (64 sequences of 8192 keys: from 50 %). 512 sequences of 128 and 256 of 512 keys have
// 16-token pages; 2000 of 300 keys 16 query and 2 key/value heads and 16-token pages;
// at d = 64, 64 sequences of 4096 keys have 64 query heads, 128 of 1000 keys 32-token
// pages. Chunks of 40 rows are over 1434-2048 keys; 8 chunks of 448 rows are not causal,
// over 1050-1500 states with 16 query and key/value heads and 128-token pages; 5 drafted
// tokens of 16 sequences have 28 query and 4 key/value heads, d = 64, fp16, 32-token
// pages and up to 4001 keys; the mixed step is 16 decoding sequences and a 512-row chunk
// of up to 4096 keys each; the chunk of 4096 rows has 128-token pages.
//
// Work split: lengths are known on the device only, and ragged, so units are not
// dealt out whole. All units lie one after another on a line, each as long as its
// visible keys plus a constant for its start and end; CTA i of the grid takes the
// i-th equal piece of the line, cut at key-tile borders. A CTA then holds part of
// at most two units that others share (its first and its last) and writes their
// partial states (m, l, divisor of o, o) to the workspace, at most two per CTA
// whatever the problem; paged_combine_kernel merges them in the order of the
// keys. Decode of a few long sequences, a single short one and a long prompt
// chunk all fill the GPU the same way, and the order of every sum is fixed.
//
// A tile's keys are copied page by page with TMA (one box per page and 64
// columns; the lanes of the producer warp each look one page up). The last tile's
// rows beyond the sequence's length are not used: scores there are masked by
// selection, and a helper warp zeroes those rows of V in shared memory before the
// P V product, since 0 * NaN from an unwritten slot would reach O.
//
// Warp roles: softmax (one thread per row; warps 0-3 of tile 0, 4-7 of tile 1 in the
// NT = 2 kernel), then K (and V) producer, MMA issuer, Q producer and V tail, and a
// fourth that produces V or issues the second tile's products. Every role finds
// the CTA's units for itself.
// Tensor memory (lane = row): S_t [128 t, +128), O_t [256 + d t, +d), and P_t in
// columns of its own [384 + 64 t, +64) except for NT = 2 at d = 128, where the
// columns run out and P_t overwrites S_t ("split P" in attn_fwd_sm103.cu has the
// reasons for either order of products).
//
// Measured and not kept: both softmax warpgroups on one tile's key columns in halves
// (no faster: one-tile units wait for their copies); separate barriers for the two Q
// tiles of a unit inside the issuer's loop (5 % slower), or a third Q tile loaded
// ahead in place of a fifth K or V tile (no faster); V by a warp of its own for pages of 64
// tokens and more (3 % slower); O transposed between lanes into whole 128-byte
// lines (as slow as the 32 rows a store touches without); the P V product begun on the
// first half of P (3 % slower: the issuer waits for one tile's second half while the
// other tile could go on); the part of a unit that an earlier CTA starts taken last, so
// that the CTAs sweep the keys in step (3 % on a 4096-row chunk over 32768 keys, but its
// longer walk costs short units up to 12 %: 512 sequences of 128 keys 69 us, 62 without;
// limited to two-tile units 2 %, and 3 % lost on a mixed step); the next part's first page
// looked up before a part's last copies (512 sequences of 128 keys 65 us, 62 without).
// Exponentials are not a bound: with 7 in 8 of them left out everything takes 92-101 %.
#pragma once
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"
#include "ptx_f8.cuh"

namespace attn {
namespace {

using namespace ptx;

constexpr int BM = 128;  // query rows per tile
constexpr int BN = 128;  // keys per tile
constexpr float kRescaleThreshold = 8.0f;
// What a unit costs beyond its key tiles, in keys: with 64 a prompt of 8192 tokens takes 400 us, with 384 it
// takes 369, and the verification of 5 drafted tokens of 16 sequences 19.3 and 18.0.
constexpr int kUnitCost = 384;
// A key tile of a two-tile unit against one of a one-tile unit: the mixed step takes 68.5 us (1.2: 72.3, 2.0:
// 70.0), at d = 64 51.7 us (54.6, 57.0).
constexpr float kPairCost = 1.5f;
// The same for kBytes, where the batch's one-tile units are small and where they are not. At d = 128 a mixed step of 64
// decoding sequences and a 512-row chunk (up to 4096 keys each) takes 154 us with 2.7 (2.0: 170, 2.4: 165, 3.0: 158, 3.5: 168;
// in fp16 160, 182, 174, 164, 174), 24 trees of 22 to 61 tokens (40 query and 8 key/value heads, up to 8192 keys) in fp16 174 us
// with 1.4 (1.2: 185, 1.3: 180, 1.6: 181), in bf16 182 (173, 175, 195). At d = 64 less would do: 157 and 148 us with 2.7 and 2.0, 144
// and 137 in fp16, 171 and 161 with 1.4 and 1.2, 168 and 158 in fp16.
constexpr float kPairCostSmall = 2.7f, kPairCostCodes = 1.4f;
constexpr unsigned kFull = 0xffffffffu;
constexpr int kIssueUnroll = 4;  // k-steps of a product in a row: 2 and 8 are within 2 %, 1 is 13 % slower

// The kernels: kFew and kOne for batches whose sequences all fit one tile, kMixed for those with longer
// chunks (there each CTA works either on one-tile or on two-tile units). With one unit in hand a CTA waits
// between its steps: for the softmax where d = 64, and from one unit to the next where keys are few. So two
// CTAs share an SM, with half of its shared and tensor memory each, where that is enough: at d = 64 (128
// sequences of 1000 keys 50 us, 59 with one CTA; 64 of 4096 keys 86 and 90), and at d = 128 for up to
// kFewRows rows if the block table has room for up to kFewKeys keys (kFew: 512 sequences of 128 keys take
// 60 us, 100 with kOne, 2000 of 300 keys 117 and 129, 256 of 512 keys 85 and 85; longer ones stream better
// with all of the SM's memory, 64 sequences of 8192 keys 239 us against 243).
enum : int { kFew = 0, kOne = 1, kMixed = 2 };
constexpr int kFewRows = 32, kFewKeys = 384;

// Variants of each: kRun attends to runs of tokens over a 16-bit cache, kTree to trees (each row has bits
// that say which of the sequence's new rows it sees), kBytes to either over a cache of E4M3 codes.
//
// The roles of kBytes and what they do are further down, with its Cfg8.
enum : int { kRun = 0, kTree = 1, kBytes = 2 };

template <int D, int KERNEL, int VAR>
struct Shape {
    static constexpr bool kF8 = VAR == kBytes;
    static constexpr int kTiles = KERNEL == kMixed ? 2 : 1;  // of a unit, at most
    static constexpr int kPerSm = !kF8 && (KERNEL == kFew || (KERNEL == kOne && D == 64)) ? 2 : 1;
    static constexpr int kFirst = 4 * kTiles;  // the first warp behind the softmax warps
    // warps of kBytes behind those: four converters, and in kOne the factors' and P V's (in kMixed those are softmax warps
    // that a CTA on one-tile units has left) up to a whole warpgroup
    static constexpr int kConverters = !kF8 ? 0 : KERNEL == kMixed ? 4 : 8;
    static constexpr int kThreads = (KERNEL == kMixed ? 384 : 256) + 32 * kConverters;
    // shared memory for Q, K and V tiles
    static constexpr int kTilesBytes = (KERNEL == kFew ? 104 : kPerSm == 2 ? 96 : 224) * 1024;
    static constexpr int kSmemBytes = kTilesBytes + 2048 + 1024;  // barriers and schedule + alignment slack
    static_assert(kPerSm * (kSmemBytes + 1024) <= 228 * 1024, "shared memory");
    static constexpr uint32_t kTmemCols = 512 / kPerSm;
    // registers per thread after the rebalance: the softmax warps hold a row of scores each
    static constexpr bool kRebalance = KERNEL == kMixed || kPerSm == 2 || kF8;
    static constexpr int kLaunchRegs = kThreads * kPerSm == 384 ? 168 : 128;
    static constexpr int kSoftmaxRegs = KERNEL != kMixed ? (kF8 ? 240 : 184) : D == 64 || kF8 ? 192 : 200;
    static constexpr int kOtherRegs = KERNEL != kMixed ? (kF8 ? 88 : 72) : kF8 ? 64 : D == 64 ? 120 : 104;
    // of kBytes, in a CTA on one-tile units: of four warps, where in kMixed the second tile's stay at the launch's
    static constexpr int kOneTileRegs = 240;
    static_assert(!kF8 || KERNEL != kMixed || 4 * kOneTileRegs + 4 * kLaunchRegs + 8 * kOtherRegs <= 16 * kLaunchRegs, "register split");
    static_assert(!kRebalance || 4 * kTiles * kSoftmaxRegs + (kThreads / 32 - 4 * kTiles) * kOtherRegs <= kThreads / 32 * kLaunchRegs,
                  "register split");
};

// A CTA of the kernel KERNEL that works on units of NT tiles.
template <int D, int NT, int KERNEL, int VAR>
struct Cfg {
    using Kernel = Shape<D, KERNEL, VAR>;
    static constexpr bool kF8 = VAR == kBytes;
    static constexpr int kBoxes = D / 64;
    static constexpr int kTileBytes = BM * D * 2;
    // P in tensor-memory columns of its own, where there are enough
    static constexpr bool kSplit = D == 64 || (NT == 1 && KERNEL != kFew);
    // One issuer for both tiles where P lies over S: the tiles' products must not mix, or their softmaxes run at
    // the same time and the tensor pipe waits for both (two issuers 20 % slower, two that take turns 2 %).
    static constexpr bool kOneIssuer = !kSplit && NT == 2;
    static constexpr int kIssuers = kOneIssuer ? 1 : NT;
    static constexpr int kQOff = 0;
    // Q tiles are loaded ahead of their unit: with one tile into as many slots as its rows leave room for, with
    // two into two more slots at d = 64 (at d = 128 a third Q tile is no faster than a fifth K or V tile)
    static constexpr int kQTiles = NT == 1 ? 1 : D == 128 ? 2 : 4;
    static constexpr int kQBytes = KERNEL == kFew ? kFewRows * D * 2 : kQTiles * kTileBytes;
    static constexpr int kKVOff = kQOff + kQBytes;
    static constexpr int kStages = (Kernel::kTilesBytes - kKVOff) / kTileBytes;  // K and V tiles in flight
    // tensor-memory columns of tile t; S_t is at BN t
    static constexpr int o_col(int t) { return KERNEL == kFew ? 128 : NT == 1 && D == 64 ? 192 : 256 + D * t; }
    static constexpr int p_col(int t) { return !kSplit ? BN * t : NT == 1 && D == 64 ? 128 : 384 + 64 * t; }
    static_assert(NT == 2 || o_col(0) + D <= (int)Kernel::kTmemCols, "tensor memory");
    // warps: K (and V) producer, MMA issuer, Q producer and V tail; the fourth is the V producer, except where
    // it has to issue the second tile's products
    static constexpr int kProducer = Kernel::kFirst, kIssuer = kProducer + 1, kTail = kProducer + 2;
    static constexpr int kFourth = kProducer + 3;
    static constexpr bool kVProducer = kIssuers == 1;
};

// A CTA of the kBytes variant that works on units of NT tiles; SMALL: one-tile units of up to 32 rows.
//
// Keys go to the tensor cores as the codes they are, since a product of E4M3 codes is exact in fp32: Q is split
// into kPieces 8-bit numbers whose sum it is (split_pair), and S is the sum of their products with the codes,
// times the key's scale and the row's. Values are widened to 16 bits by converter warps, scales included. P in 8-bit
// pieces, which would need no converters, is slower: the splitting comes on top of the softmax, which a tile then waits
// for.
//
// Widening keys and values, with Q as it is, took 335 us for 64 sequences of 8192 keys: the converters' integer
// instructions issue at 64 lanes a cycle.
template <int D, bool F16, int NT, int KERNEL, bool SMALL>
struct Cfg8 {
    using Kernel = Shape<D, KERNEL, kBytes>;
    static constexpr int kTileBytes = BN * D;      // of codes
    static constexpr int kPieces = F16 ? 3 : 2;    // of 4, 3 and 3 bits of Q's 11 or 8 (split_pair)
    // Tensor memory of units of one tile: scores from 0 on, Q's pieces (a product then reads keys alone from shared
    // memory), O, and P of two tiles in turn. Units of two tiles have no room for Q there.
    static constexpr bool kQTmem = NT == 1;
    static constexpr int kQCol = 128, kOCol = 256, kPCol = 384;
    static constexpr int kQBytes = kQTmem ? 0 : NT * kPieces * kTileBytes;
    // widened values, then rings of codes and of their scales, and the keys' factors as floats
    static constexpr int kWide = D == 128 ? 2 : 3;
    static constexpr int kWideOff = kQBytes, kKeyOff = kWideOff + kWide * 2 * kTileBytes;
    // small units: pieces of Q and factors of its rows for two units, and where copies of rows are merged
    static constexpr int kQSlots = 2, kQPitch = D + 16, kQSlot = 32 * kPieces * kQPitch + 32 * 4;
    static constexpr int kStateBytes = 4 * 32 * 16, kMergeBytes = 4 * 32 * 36 * 4;
    static constexpr int kExtraBytes = SMALL ? kQSlots * kQSlot + kStateBytes + kMergeBytes : 0;
    static constexpr int kRoom = Kernel::kTilesBytes - kKeyOff - kExtraBytes;
    // Factors of a tile: the keys' scales, times 2^-bias. Two stages more than keys have: a tile of keys arrives when the products
    // with the one kKeys before it are done, and by then the softmax has read the factors of what came two before that
    // (a thread reads a tile's factors before it takes the next one's scores).
    static constexpr int kFactorBytes = BN * 4;
    static constexpr int kFit = (kRoom - 3 * kFactorBytes) / (kTileBytes + BN + kFactorBytes / 2);
    static constexpr int kBoth = kFit < 16 ? kFit : 16;
    static constexpr int kKeys = (kBoth + 1) / 2, kValues = kBoth / 2;  // stages
    static constexpr int kValueOff = kKeyOff + kKeys * kTileBytes;
    static constexpr int kKeyScaleOff = kValueOff + kValues * kTileBytes, kValueScaleOff = kKeyScaleOff + kKeys * BN;
    static constexpr int kFactors = kKeys + 2;
    static constexpr int kFactorOff = kValueScaleOff + kValues * BN;
    static constexpr int kQSlotOff = kFactorOff + kFactors * kFactorBytes;
    static constexpr int kStateOff = kQSlotOff + kQSlots * kQSlot, kMergeOff = kStateOff + kStateBytes;
    static_assert(kValues >= 1 && kQSlotOff + kExtraBytes <= Kernel::kTilesBytes, "shared memory");
    static_assert(kQCol + kPieces * D / 4 <= kOCol && kOCol + D <= kPCol, "tensor memory");
    static constexpr int kMakers = 4;  // converter warps
};

struct PagedDev {
    int B, G, Hkv, T;
    int tok_tile;     // tokens of a tile: its rows are tok_tile * G
    int num_pages, page_size, shift, max_pages;
    int causal;
    float c;          // scale * log2(e); of kBytes times 2^bias
    const int32_t *cu_q, *kv_len, *table;
    long long table_stride;
    uint8_t* o;
    float* lse;
    long long o_sr, o_sh;  // elements
    int o_wide;       // rows of o are 32-byte aligned
    float* part;      // [grid][2][NT] records of tok_tile * G rows: see record()
    int4* meta;       // [grid][2]: see below
    int* err;
    unsigned long long timeout_ns;
    int stall_after;  // test hook: the K and V producers stop after this many key tiles (0 = off)
    // kTree and kBytes: bits of the new rows that a row sees (NULL without trees). Sequences of more than
    // tree_nodes rows are causal; without trees that is 0 for a causal call and no limit otherwise.
    const uint32_t* tree;
    long long tree_stride;
    int tree_words, tree_nodes;
    float key_bias;   // kBytes: 2^-bias, which goes onto the keys' scales (key_bias_of)
    // kBytes: scales of keys and values, and their strides over (page, head)
    const uint8_t *k_scale, *v_scale;
    long long ks_page, ks_head, vs_page, vs_head;
    const uint16_t* q;
    long long q_sr, q_sh;  // elements
};

// What the combine kernel reads about a CTA's slot: x = 0 nothing, 1 a part, 2 the unit's last part;
// y = first query row of the unit, z = its tokens, w = key/value head.
enum : int { kNone = 0, kPart = 1, kLast = 2 };

struct Seq {
    int row0, n, len;  // first row of q, rows, keys; within the arrays whatever the lengths say
};

// Where a warp's walk over its CTA's units stands: the unit to come.
struct Place {
    long long u0;    // where it starts on the line
    int b, h, blk;   // sequence, key/value head, number of the unit in them
    Seq seq;
};

struct __align__(16) Shared {
    uint64_t q_full[4], q_empty[4];  // of the Q slots, which are used in turn
    uint64_t kv_full[13], kv_empty[13], v_tail[13];
    // kBytes: codes fetched, of keys their factors made, released; kv_full and kv_empty are the widened values'
    uint64_t k_full[8], k_ready[8], k_empty[8], v_full[8], v_empty[8];
    uint64_t s_full[2], p_full[2], o_full[2], s_free[2], pv_done[2];
    uint64_t drain[2], merged;
    long long x0, x1;      // this CTA's piece of the line
    Place first;           // the unit that holds x0; u0 = -1 if there is none
    Place place[16];       // of each warp
    int4 unit[8];          // of each softmax warp, the unit it is in: first row of q, tokens, key/value
                           // head, 1 if it holds the first key tile + 2 if the last
    long long scan[2][16]; // per warp: its sequences' cost on either line
    int pair;              // whether this CTA works on two-tile units
    int widest[16], most_rows, sm_warps;  // most rows of a one-tile unit; softmax warps of a tile that hold rows
    uint32_t issued[2];    // ring items issued: of K (even numbers) all below the first, of V all below the second
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(Shared) <= 2048, "barrier area");

// ---------------------------------------------------------------- the line of units
__device__ __forceinline__ Seq seq_of(const PagedDev& p, int b, bool* bad) {
    const int c0 = p.cu_q[b], c1 = p.cu_q[b + 1], len = p.kv_len[b];
    const long long most = (long long)p.max_pages << p.shift;
    Seq s;
    s.row0 = min(max(c0, 0), p.T);
    s.n = min(max(c1, s.row0), p.T) - s.row0;
    s.len = (int)min((long long)max(len, 0), most);
    if (bad) *bad |= c0 < 0 || c1 < c0 || c1 > p.T || len < 0 || len > most || (b == 0 && c0 != 0);
    return s;
}

template <int VAR>
__device__ __forceinline__ bool is_causal(const PagedDev& p, const Seq& s) {
    return VAR == kRun ? p.causal : s.n > p.tree_nodes;
}

// Keys that the last of a sequence's first `tok` rows sees (of a tree's, may see).
template <int VAR>
__device__ __forceinline__ int visible(const PagedDev& p, const Seq& s, int tok) {
    return is_causal<VAR>(p, s) ? max(0, s.len - s.n + tok) : s.len;
}

// Cost of the first i units of one head (all but the sequence's last unit are full, so their visible
// keys grow by `step` rows each, from where they are positive on).
template <int VAR>
__device__ __forceinline__ long long cost_before(const PagedDev& p, const Seq& s, int step, long long i) {
    if (!is_causal<VAR>(p, s)) return i * (s.len + kUnitCost);
    const long long base = s.len - s.n;
    const long long m = base >= 0 ? 1 : -base / step + 1;  // the first unit (from 1) with a visible key
    long long sum = i * kUnitCost;
    if (i >= m) sum += (i - m + 1) * base + step * (i * (i + 1) / 2 - m * (m - 1) / 2);
    return sum;
}

template <int VAR>
__device__ __forceinline__ long long head_cost(const PagedDev& p, const Seq& s, int step) {
    if (s.n == 0) return 0;
    const int units = (s.n + step - 1) / step;
    return cost_before<VAR>(p, s, step, units - 1) + visible<VAR>(p, s, s.n) + kUnitCost;
}

// Whether a sequence is worked on in two-tile units: in the kernel that has them, if one tile does not
// hold its rows.
template <int NT>
__device__ __forceinline__ bool is_pair(const PagedDev& p, const Seq& s) {
    return NT == 2 && s.n > p.tok_tile;
}

// Finds this CTA's piece of the line. All threads take part. In the NT = 2 kernel there are two lines, of
// one-tile and of two-tile units, and the CTAs are shared out between them by their costs: the former are
// bound by reading keys and values, the latter by the tensor cores, so they run side by side.
template <int NT, int THREADS, int VAR>
__device__ __forceinline__ void locate(const PagedDev& p, Shared& sh) {
    constexpr int WARPS = THREADS / 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    bool bad = false;
    long long done[2] = {0, 0};  // cost of the chunks of sequences before this one, of either line
    int rows = 0;
    // the last chunk: this thread's sequence, its cost per head, and the lines' ends behind it
    Seq s{0, 0, 0};
    long long per_head = 0, end[2] = {0, 0};
    auto scan = [&](int b0, bool first) {
        const int b = b0 + tid;
        s = Seq{0, 0, 0};
        if (b < p.B) s = seq_of(p, b, first ? &bad : nullptr);
        const bool two = is_pair<NT>(p, s);
        per_head = head_cost<VAR>(p, s, two ? 2 * p.tok_tile : p.tok_tile);
        if (first && !two) rows = max(rows, min(s.n, p.tok_tile) * p.G);
#pragma unroll
        for (int k = 0; k < NT; ++k) {
            long long x = two == (k == 1) ? per_head * p.Hkv : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(kFull, x, o);
                if (lane >= o) x += u;
            }
            end[k] = done[k] + x;
            if (lane == 31) sh.scan[k][warp] = x;
        }
        if (first) {
            const int widest = __reduce_max_sync(kFull, rows);
            if (lane == 0) sh.widest[warp] = widest;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < NT; ++k) {
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                if (w < warp) end[k] += sh.scan[k][w];
                done[k] += sh.scan[k][w];
            }
        }
    };
    if (tid == 0) sh.first.u0 = -1;
    for (int b0 = 0; b0 < p.B; b0 += THREADS) {
        if (b0 > 0) __syncthreads();  // the last use of scan
        scan(b0, true);
    }
    if (bad && blockIdx.x == 0) atomicCAS(p.err, 0, ATTN_ERR_INVALID);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) rows = max(rows, sh.widest[w]);
    int i = blockIdx.x, n = gridDim.x;
    bool pair = false;
    if (NT == 2) {
        const float pair_cost = VAR != kBytes ? kPairCost : rows <= 32 ? kPairCostSmall : kPairCostCodes;
        const float c0 = (float)done[0], c1 = (float)done[1] * pair_cost;
        int n0 = done[0] == 0 ? 0 : max(1, (int)(n * (c0 / (c0 + c1)) + 0.5f));
        if (done[1] > 0) n0 = min(n0, n - 1);
        // An even number of kBytes' CTAs, as far as one may judge by times: pairs of CTAs seem to share a cache of instructions
        // that the loops of one kind fill, so that a pair of both kinds falls behind (24 trees 174 us, 190 with any number; a mixed
        // step 154 and 185). Which SM a CTA comes to is not promised; nothing but time depends on it.
        if (VAR == kBytes && n0 > 1) n0 &= ~1;
        pair = i >= n0;
        i = pair ? i - n0 : i;
        n = pair ? n - n0 : n0;
    }
    const long long total = pair ? done[1] : done[0];
    const long long each = total / max(n, 1), rest = total - each * n;
    const long long x0 = each * i + min((long long)i, rest), x1 = x0 + each + (i < rest ? 1 : 0);
    done[0] = done[1] = 0;
    for (int b0 = 0; b0 < p.B && x0 < x1; b0 += THREADS) {
        if (p.B > THREADS) {  // else the scan above is the one to look at
            __syncthreads();
            scan(b0, false);
        }
        const long long hi_end = pair ? end[1] : end[0];
        const long long begin = hi_end - (is_pair<NT>(p, s) == pair ? per_head * p.Hkv : 0);
        if (begin <= x0 && x0 < hi_end) {
            const int step = pair ? 2 * p.tok_tile : p.tok_tile;
            const int h = (int)((x0 - begin) / per_head);
            const long long in_head = x0 - begin - h * per_head;
            int lo = 0, hi = (s.n + step - 1) / step;  // the last unit that starts at or before in_head
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cost_before<VAR>(p, s, step, mid) <= in_head)
                    lo = mid;
                else
                    hi = mid;
            }
            sh.first = Place{begin + h * per_head + cost_before<VAR>(p, s, step, lo), b0 + tid, h, lo, s};
        }
        if ((pair ? done[1] : done[0]) > x0) break;
    }
    if (tid == 0) {
        sh.x0 = x0;
        sh.x1 = x1;
        sh.pair = pair;
        sh.most_rows = rows;
        sh.sm_warps = max(1, ((pair ? p.tok_tile * p.G : rows) + 31) / 32);
    }
}

struct Unit {
    int h, row0, ntok;  // key/value head, first row of q, tokens
    int base;           // position of the first token (causal), or the last key for all rows
    int len;            // keys of the sequence
    int b;
    int k0, cnt0, cnt1, cnt_max;  // first key tile of this part, key tiles of either tile in it
    bool first, last;   // this part holds the unit's first / last key tile
    bool causal;
    int ctx;            // keys before the sequence's new rows
    __device__ __forceinline__ int cnt(int t) const { return t == 0 ? cnt0 : cnt1; }
};

// Walks this CTA's units of NT tiles in order. Every warp role walks for itself and finds the same units;
// its place is kept in shared memory, since the softmax warps need their registers for a row of scores.
// In the mixed kernel sequences of the other kind are passed over.
template <int NT, int KERNEL, int VAR>
struct Walk {
    const PagedDev& p;
    const Shared& sh;
    Place& place;

    __device__ __forceinline__ Walk(const PagedDev& p_, Shared& sh_)
        : p(p_), sh(sh_), place(sh_.place[threadIdx.x >> 5]) {
        if ((threadIdx.x & 31) == 0) {
            place = sh.first;
            if (place.u0 < 0) place.u0 = sh.x1;
        }
    }
    // All lanes of a warp, converged.
    __device__ __forceinline__ bool next(Unit& w) {
        const int step = NT * p.tok_tile;
        const long long x0 = sh.x0, x1 = sh.x1;
        __syncwarp();
        Place at = place;
        bool mine = false;
        while (!mine && at.u0 < x1) {
            const Seq s = at.seq;
            const int tok0 = at.blk * step;
            w.ntok = min(step, s.n - tok0);
            const int keys = visible<VAR>(p, s, tok0 + w.ntok);
            const int tiles = (keys + BN - 1) / BN;
            const long long end = at.u0 + keys + kUnitCost;
            const int k0 = x0 <= at.u0 ? 0 : min(tiles, (int)((x0 - at.u0 + BN / 2) / BN));
            const int k1 = x1 >= end ? tiles : min(tiles, (int)((x1 - at.u0 + BN / 2) / BN));
            mine = k0 < k1 || (tiles == 0 && at.u0 >= x0);
            w.b = at.b;
            w.h = at.h;
            w.row0 = s.row0 + tok0;
            w.len = s.len;
            w.causal = is_causal<VAR>(p, s);
            w.ctx = s.len - s.n;
            w.base = w.causal ? s.len - s.n + tok0 : s.len - 1;
            w.k0 = k0;
            w.first = k0 == 0;
            w.last = k1 == tiles;
            w.cnt_max = k1 - k0;
            w.cnt0 = w.cnt_max;
            w.cnt1 = 0;
            if (NT == 2 && w.ntok > p.tok_tile) {  // causal: tile 0's rows may see fewer tiles
                w.cnt1 = w.cnt_max;
                w.cnt0 = max(0, min(k1, (visible<VAR>(p, s, tok0 + p.tok_tile) + BN - 1) / BN) - k0);
            }
            at.u0 = end;
            if (tok0 + step < s.n) {
                ++at.blk;
            } else {
                at.blk = 0;
                if (++at.h == p.Hkv) {
                    at.h = 0;
                    do {
                        if (++at.b >= p.B) {
                            at.u0 = x1;
                            break;
                        }
                        at.seq = seq_of(p, at.b, nullptr);
                    } while (at.seq.n == 0 || (KERNEL == kMixed && is_pair<2>(p, at.seq) != (NT == 2)));
                }
            }
        }
        __syncwarp();
        if ((threadIdx.x & 31) == 0) place = at;
        return mine;
    }
};

// The record of tile t of a CTA's slot: per row (m, l, divisor of o, unused), then o by groups of four
// columns, each group's rows side by side, so that neighbouring threads (rows) write neighbouring 16 bytes.
__device__ __forceinline__ float4* record(float* part, int slot, int tiles, int t, int rows, int d) {
    return reinterpret_cast<float4*>(part) + ((long long)slot * tiles + t) * rows * (1 + d / 4);
}

// LSE of a row from its reference maximum and sum: -inf where it has no key (sum 0), NaN where the sum is.
__device__ __forceinline__ float row_lse(float m, float l) { return l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2; }

// ---------------------------------------------------------------- helpers of the roles
__device__ __forceinline__ uint64_t step_desc(uint64_t d, uint32_t by) {
    return (d & 0xffffffff00000000ull) | ((uint32_t)d + by);
}
// Descriptors of a tile's first k-step, and the steps to the others: 16-byte units added to the start
// address, which sits in the low bits and does not overflow them. `half`: bytes from one 64-column box of a
// K-major tile to the next.
__device__ __forceinline__ uint64_t kmajor_desc(uint32_t tile) { return sdesc_sw128(tile, 16, 1024); }
__device__ __forceinline__ uint64_t kmajor_step(uint64_t d, int kk, uint32_t half) {
    return step_desc(d, (kk >> 2) * (half >> 4) + (kk & 3) * 2);
}
__device__ __forceinline__ uint64_t vmajor_desc(uint32_t tile) { return sdesc_sw128(tile, BN * 128, 1024); }
__device__ __forceinline__ uint64_t vmajor_step(uint64_t d, int kk) { return step_desc(d, kk * (16 * 128 >> 4)); }
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity, uint64_t timeout_ns) {
    const uint32_t a = smem_u32(bar);
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(a, parity))
        if (globaltimer() - t0 > timeout_ns) break;
}

// Which of four barriers have completed the given phases, for a whole converged warp. Looking at a barrier
// takes some 130 cycles, ready or not, and an issuer looks at four a key tile (4096 rows over 32768 keys 1305 us
// one after another, 1268 with this).
__device__ __forceinline__ unsigned look(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, uint64_t* c, uint32_t pc,
                                         uint64_t* d, uint32_t pd) {
    const unsigned ra = mbar_test(a, pa), rb = mbar_test(b, pb), rc = mbar_test(c, pc), rd = mbar_test(d, pd);
    return __reduce_and_sync(kFull, ra | rb << 1 | rc << 2 | rd << 3);
}

// One store of 32 bytes (sm_100 on): the epilogue's threads hold a row each, and every store instruction
// touches 32 rows whatever its width (eight prompts of 1024 tokens 85 us, 89 with 16-byte stores).
__device__ __forceinline__ void store32(void* dst, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// The page that holds key `key` for this lane: its number, or num_pages (a row of zeros to TMA) for
// one that the cache does not have.
__device__ __forceinline__ int page_at(const PagedDev& p, int b, int key, bool* bad) {
    const int page = p.table[b * p.table_stride + (key >> p.shift)];
    if (page >= 0 && page < p.num_pages) return page;
    *bad = true;
    return p.num_pages;
}

// The Q slot to come, and the phase of its uses.
struct QRing {
    uint32_t slots, at = 0, phase = 0;
    __device__ __forceinline__ explicit QRing(uint32_t n) : slots(n) {}
    __device__ __forceinline__ void next() {
        if (++at == slots) {
            at = 0;
            phase ^= 1;
        }
    }
};

// Waits for the last item issued into each slot (none was issued over one that had not landed). Out of line: short
// units run the kernel's code cold, and what they never use costs them its place (512 sequences of 128 keys 59 us, 61
// with it inline).
__device__ __noinline__ void drain_ring(Shared& bar, uint32_t stages, uint64_t timeout_ns) {
    const uint32_t end = max(bar.issued[0], bar.issued[1]);
    for (uint32_t s = 0; s < stages && s < end; ++s) {
        uint32_t i = s + (end - 1 - s) / stages * stages;
        while (i >= bar.issued[i & 1] && i >= stages) i -= stages;
        if (i < bar.issued[i & 1]) drain_wait(&bar.kv_full[s], (i / stages) & 1, timeout_ns);
    }
}

// ---------------------------------------------------------------- trees
// Bits of the 32 N keys from key0 on that a row sees, whose words are at `row` (NULL: none of the new rows).
template <int N>
__device__ __forceinline__ void tree_bits(const PagedDev& p, const uint32_t* row, int key0, int ctx, int len, uint32_t (&bits)[N]) {
    const int rel = key0 - ctx;  // of the first key among the new rows'
    const int at = rel >> 5;
    uint32_t w[N + 1];
#pragma unroll
    for (int k = 0; k <= N; ++k) w[k] = at + k < 0 ? ~0u : at + k < p.tree_words && row ? row[at + k] : 0u;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        bits[k] = __funnelshift_r(w[k], w[k + 1], rel & 31);
        const int held = len - key0 - 32 * k;
        if (held < 32) bits[k] &= held <= 0 ? 0u : (1u << held) - 1;
    }
}

// ---------------------------------------------------------------- 8-bit caches
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// The two fp16 numbers of x times that in the lower half of y, in fp32.
__device__ __forceinline__ float2 widen2(uint32_t x, uint32_t y) {
    float2 d;
    asm("{\n\t.reg .b16 lo, hi, f, g;\n\tmov.b32 {lo, hi}, %2;\n\tmov.b32 {f, g}, %3;\n\t"
        "fma.rn.f32.f16 %0, lo, f, 0f00000000;\n\tfma.rn.f32.f16 %1, hi, f, 0f00000000;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "r"(x), "r"(y));
    return d;
}

// 16 codes as fp16 numbers.
__device__ __forceinline__ void codes16(uint4 v, uint32_t (&out)[8]) {
    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(out[k]) : "h"((uint16_t)(in[k / 2] >> (16 * (k & 1)))));
}

// 16 codes times the scale 2^(s - 127), which fp16 has to hold (2^-24 to 2^15): the codes as fp16 numbers, times the
// scale in fp16, or for bf16 in fp32, exact, by multiply-adds of fp16 numbers into fp32. NaN stays NaN on the way.
// Moving a code's bits to where bf16 has them takes as many instructions (a byte permutation that repeats the sign, a
// move, a mask, a multiplication), but turns NaN into 480, and is hardly faster: decode of 64 sequences of 8192 keys takes
// 160 us, 161 in that way, 187 with a look for NaN codes on top.
template <bool F16>
__device__ __forceinline__ void widen16(uint4 v, int s, uint32_t (&out)[8]) {
    const float scale = __uint_as_float((uint32_t)s << 23);
    const uint32_t f = pack_f16(scale, scale);
    codes16(v, out);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if constexpr (F16) {
            out[k] = mul2(out[k], f);
        } else {
            const float2 x = widen2(out[k], f);
            out[k] = pack_bf16(x.x, x.y);
        }
    }
}

// The same for any scale (in bf16, bytes 0 and 255 are 2^-127 and NaN): in two multiplications where fp16 has to hold the
// factors. Whatever is left of a scale beyond 2^30 would only come upon values beyond fp16's range.
template <bool F16>
__device__ __forceinline__ void widen16_any(uint4 v, int s, uint32_t (&out)[8]) {
    codes16(v, out);
    if constexpr (F16) {
        const int s0 = min(max(s, 113), 142), s1 = min(127 + s - s0, 142);
        const float scale = __uint_as_float((uint32_t)s0 << 23), rest = __uint_as_float((uint32_t)s1 << 23);
        const uint32_t f = pack_f16(scale, scale), more = pack_f16(rest, rest);
#pragma unroll
        for (int k = 0; k < 8; ++k) out[k] = mul2(mul2(out[k], f), more);
    } else {
        const float scale = __uint_as_float(s == 0 ? 0x00400000u : s == 255 ? 0x7fc00000u : (uint32_t)s << 23);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float2 x = unpack_h16<true>(out[k]);
            out[k] = pack_bf16(x.x * scale, x.y * scale);
        }
    }
}

// Makes the share of warp c of W of a 16-bit tile from a tile of codes: rows of 128 bytes per 64 columns, 16-byte
// chunks swizzled by the row as TMA does. Rows from `left` on become 0. A warp takes every W-th group of 8 rows.
// A lane has 16 codes of a row at a time, and the same row of every group and the same columns in all of its turns,
// so that its addresses differ by constants. Eight lanes that access memory together read and write all
// banks: at d = 128 (codes swizzled like the tile) four lanes on the first columns of a row and four on those of
// the row that differs in bits 0 and 2, at d = 64 four on each of two rows.
// The roles of a CTA share its instruction cache. LOOP: the two turns in a loop, for the kernel that has both kinds of unit (a
// mixed step of 64 sequences and a chunk 154 us, 183 unrolled); where units are of one tile, both at once (64 sequences of 8192
// keys 160 us, 169 in a loop; 2000 of 300 keys 251 and 241).
template <int D, bool F16, int W, bool LOOP>
__device__ __forceinline__ void widen_tile(const uint8_t* raw, const uint8_t* scale, uint8_t* tile, int left, int c, int lane) {
    constexpr int kTurns = D == 128 ? 2 : 1;  // for 8 rows
    constexpr int kEach = BN / 8 / W;         // groups of a warp
    static_assert(kEach * 8 * W == BN, "groups");
    const int ch = D == 128 ? (lane & 3) | (lane & 8) >> 1 : lane & 3;
    const int r0 = D == 128 ? (lane >> 4) ^ (lane & 4 ? 5 : 0) : lane >> 2;
    // scales that widen16 does not take are looked for once a tile
    const uint32_t s4 = *reinterpret_cast<const uint32_t*>(scale + lane * 4);
    const bool other = (__vcmpltu4(s4, 0x67676767u) | __vcmpgtu4(s4, 0x8e8e8e8eu)) != 0;
    // a turn's first row, and of a row: where its codes are, and where the two chunks go
    auto row_of = [&](int turn) { return c * 8 + (r0 ^ (turn * 2)); };
    auto codes_of = [&](int row) { return raw + row * D + (D == 128 ? (ch ^ (row & 7)) * 16 : ch * 16); };
    auto chunk_of = [&](int row, int k) { return tile + (ch >> 2) * BN * 128 + row * 128 + (((ch & 3) * 2 + k) ^ (row & 7)) * 16; };
    if (!__any_sync(kFull, other) && left >= BN) {
#pragma unroll LOOP ? 1 : kTurns
        for (int turn = 0; turn < kTurns; ++turn) {
            const int row = row_of(turn);
            const uint8_t* from = codes_of(row);
            uint8_t *to0 = chunk_of(row, 0), *to1 = chunk_of(row, 1);
            uint4 v[kEach];
            int s[kEach];
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                v[i] = *reinterpret_cast<const uint4*>(from + i * W * 8 * D);
                s[i] = scale[row + i * W * 8];
            }
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                uint32_t out[8];
                widen16<F16>(v[i], s[i], out);
                *reinterpret_cast<uint4*>(to0 + i * W * 1024) = make_uint4(out[0], out[1], out[2], out[3]);
                *reinterpret_cast<uint4*>(to1 + i * W * 1024) = make_uint4(out[4], out[5], out[6], out[7]);
            }
        }
    } else {
#pragma unroll 1
        for (int turn = 0; turn < kTurns; ++turn) {
#pragma unroll 1
            for (int row = row_of(turn); row < BN; row += W * 8) {
                uint32_t out[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                if (row < left) widen16_any<F16>(*reinterpret_cast<const uint4*>(codes_of(row)), scale[row], out);
                *reinterpret_cast<uint4*>(chunk_of(row, 0)) = make_uint4(out[0], out[1], out[2], out[3]);
                *reinterpret_cast<uint4*>(chunk_of(row, 1)) = make_uint4(out[4], out[5], out[6], out[7]);
            }
        }
    }
}

// Two values of Q over the row's factor (at most 3584) as sums of 8-bit numbers: an E4M3 number (4 bits, up to 448) and one
// (bf16) or two (fp16) E5M2 numbers (3 bits). Up to 448 the nearest E4M3 number leaves at most 8 units of a bf16 value's 8
// bits, which 3 bits hold; of an fp16 value's 11 bits it leaves up to 64 units, of which an E5M2 number leaves up to 4.
// Beyond 448 the nearest E5M2 number comes first and leaves at most 256, 16 (fp16: 128) units, of which an E4M3 number leaves
// none (4). All exact from 2^-6 on, E4M3's least normal number; below, it leaves up to 2^-10, and the error is at most 2^-14
// (fp16: 2^-17), which is 2^-24 (2^-27) of the row's largest value.
template <bool F16>
__device__ __forceinline__ void split_pair(uint32_t x, float f, uint16_t& a, uint16_t& b, uint16_t& c) {
    const float2 y2 = fmul2(unpack_h16<F16>(x), make_float2(f, f));
    uint32_t y = pack_f16(y2.x, y2.y), large, back;
    asm("{\n\t.reg .b32 m;\n\tabs.f16x2 m, %1;\n\tset.gt.u32.f16x2 %0, m, %2;\n\t}" : "=r"(large) : "r"(y), "r"(0x5f005f00u));
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(b) : "r"(y));
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(back) : "h"(b));
    const uint32_t first = back & large;
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(y) : "r"(first));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(a) : "r"(y));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(a));
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(y) : "r"(back));
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(b) : "r"(first | (y & ~large)));
    if constexpr (F16) {
        asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(back) : "h"(b));
        asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(y) : "r"(back & ~large));
        asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(c) : "r"(y));
    }
}

// The smallest e with top <= 3584 * 2^e, 3584 = 1.75 * 2^11, as far as the factor 2^-e is a plain number.
constexpr int kMostRowExponent = 116;
__device__ __forceinline__ int row_exponent(float top) {
    const uint32_t bits = __float_as_uint(top);
    return min(max((int)(bits >> 23) - 138 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0), -119), kMostRowExponent);
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// What a row whose largest magnitude is `top` is multiplied by before it is split, with e = row_exponent(top). The 8-bit
// formats saturate: a row with an infinity becomes NaN instead, so that it shows in O and LSE.
__device__ __forceinline__ float split_factor(float top, int e) { return top < INFINITY ? pow2f(-e) : NAN; }

// The largest magnitude of 16-bit values, two at a time.
template <bool F16>
__device__ __forceinline__ void take_max(uint32_t& top, uint32_t x) {
    const uint32_t mag = x & 0x7fff7fffu;
    if constexpr (F16)
        asm("max.f16x2 %0, %0, %1;" : "+r"(top) : "r"(mag));  // a NaN does not count
    else
        asm("max.bf16x2 %0, %0, %1;" : "+r"(top) : "r"(mag));
}

// tmem_st16 for 8 columns.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Splits a thread's row of Q (NULL: a row that nobody reads) into the pieces of its tile, in tensor memory at `tmem` or
// in shared memory at `tile` as row r of K-major tiles, and returns the row's factor 2^e. Reads the row twice, and splits 32
// columns at a time in a loop: the roles of a CTA share its instruction cache, and a row in registers costs spills.
template <int D, bool F16, bool TMEM>
__device__ __forceinline__ float split_row(const uint16_t* src, uint32_t tmem, uint8_t* tile, int r) {
    constexpr int kPieces = F16 ? 3 : 2;
    const uint4* words = reinterpret_cast<const uint4*>(src);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
        const uint4 v = src ? words[i] : make_uint4(0, 0, 0, 0);
        take_max<F16>(top, v.x), take_max<F16>(top, v.y), take_max<F16>(top, v.z), take_max<F16>(top, v.w);
    }
    const float2 t2 = unpack_h16<F16>(top);
    const float largest = fmaxf(t2.x, t2.y);
    const int e = row_exponent(largest);
    const float f = split_factor(largest, e);
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t out[kPieces][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 v = src ? words[c0 / 8 + i] : make_uint4(0, 0, 0, 0);
            const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint16_t a[2], b[2], c[2] = {0, 0};
#pragma unroll
                for (int k = 0; k < 2; ++k) split_pair<F16>(x[2 * j + k], f, a[k], b[k], c[k]);
                out[0][2 * i + j] = a[0] | (uint32_t)a[1] << 16;
                out[1][2 * i + j] = b[0] | (uint32_t)b[1] << 16;
                if constexpr (F16) out[kPieces - 1][2 * i + j] = c[0] | (uint32_t)c[1] << 16;
            }
        }
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            if constexpr (TMEM) {
                tmem_st8(tmem + (k * D + c0) / 4, out[k]);
            } else {
                uint8_t* dst = tile + k * BM * D + r * D;
                const int sw = D == 128 ? r & 7 : (r >> 1) & 3;
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    *reinterpret_cast<uint4*>(dst + (((c0 / 16 + i) ^ sw) << 4)) =
                        make_uint4(out[k][4 * i], out[k][4 * i + 1], out[k][4 * i + 2], out[k][4 * i + 3]);
            }
        }
    }
    if constexpr (TMEM) {
        tmem_wait_st();
        tc_fence_before();
    } else {
        fence_proxy_async_smem();
    }
    return pow2f(e);
}

// The same by a warp for the first rows of a unit, pieces and factors in shared memory at `slot`: lanes side by side
// hold four columns of a row.
template <int D, bool F16, int PITCH>
__device__ __forceinline__ void split_unit(const PagedDev& p, const Unit& w, uint8_t* slot, int lane) {
    constexpr int kPieces = F16 ? 3 : 2, kLanes = D / 4, kAtOnce = 32 / kLanes;
    float* factors = reinterpret_cast<float*>(slot + 32 * kPieces * PITCH);
    const int rows = w.ntok * p.G, col = lane % kLanes;
    for (int r0 = 0; r0 < rows; r0 += 4 * kAtOnce) {
        uint2 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + i * kAtOnce + lane / kLanes;
            x[i] = make_uint2(0, 0);
            if (r < rows)
                x[i] = *reinterpret_cast<const uint2*>(p.q + (w.row0 + r / p.G) * p.q_sr + (w.h * p.G + r % p.G) * p.q_sh + col * 4);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + i * kAtOnce + lane / kLanes;
            uint32_t top = 0;
            take_max<F16>(top, x[i].x);
            take_max<F16>(top, x[i].y);
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1) take_max<F16>(top, __shfl_xor_sync(kFull, top, o));
            const float2 t2 = unpack_h16<F16>(top);
            const float largest = fmaxf(t2.x, t2.y);
            const int e = row_exponent(largest);
            const float f = split_factor(largest, e);
            uint16_t a[2], b[2], c[2] = {0, 0};
            split_pair<F16>(x[i].x, f, a[0], b[0], c[0]);
            split_pair<F16>(x[i].y, f, a[1], b[1], c[1]);
            if (r < rows) {
                uint8_t* dst = slot + r * PITCH + col * 4;
                *reinterpret_cast<uint32_t*>(dst) = a[0] | (uint32_t)a[1] << 16;
                *reinterpret_cast<uint32_t*>(dst + 32 * PITCH) = b[0] | (uint32_t)b[1] << 16;
                if constexpr (F16) *reinterpret_cast<uint32_t*>(dst + 64 * PITCH) = c[0] | (uint32_t)c[1] << 16;
                if (col == 0) factors[r] = pow2f(e);
            }
        }
    }
}

// What a row's scores are multiplied by behind their keys' factors: c * 2^e. Above 0, so that masked scores stay -inf.
__device__ __forceinline__ float row_factor(float c, float f) { return fmaxf(c * f, FLT_MIN); }

// Descriptor of a K-major tile of codes: rows of 128 bytes with the 128-byte swizzle, or of 64 with the 64-byte one
// (layout 4). A product's k-step is 32 codes.
template <int D>
__device__ __forceinline__ uint64_t codes_desc(uint32_t tile) {
    if constexpr (D == 128) return sdesc_sw128(tile, 16, 1024);
    return (sdesc_sw128(tile, 16, 512) & ~((uint64_t)7 << 61)) | ((uint64_t)4 << 61);
}

// drain_ring for the rings of codes.
__device__ __noinline__ void drain_codes(Shared& bar, uint32_t keys, uint32_t values, uint64_t timeout_ns) {
    for (uint32_t s = 0; s < keys && s < bar.issued[0]; ++s)
        drain_wait(&bar.k_full[s], ((bar.issued[0] - 1 - s) / keys) & 1, timeout_ns);
    for (uint32_t s = 0; s < values && s < bar.issued[1]; ++s)
        drain_wait(&bar.v_full[s], ((bar.issued[1] - 1 - s) / values) & 1, timeout_ns);
}

// The factors of one-tile units' keys, by a warp of its own: the products with keys do not wait for values to be widened
// then.
template <int D, bool F16, int KERNEL, bool SMALL>
__device__ __forceinline__ void make_factors(const PagedDev& p, uint8_t* smem, Shared& bar) {
    using E = Cfg8<D, F16, 1, KERNEL, SMALL>;
    const int lane = threadIdx.x & 31;
    const WaitCtl wc{p.err, &bar.abort_flag, p.timeout_ns};
    Walk<1, KERNEL, kBytes> walk(p, bar);
    Unit w;
    uint32_t n = 0;
    bool ok = true;
    while (ok && walk.next(w)) {
        for (int j = 0; j < w.cnt_max && ok; ++j, ++n) {
            const uint32_t s = n % E::kKeys;
            ok = mbar_wait_warp(&bar.k_full[s], (n / E::kKeys) & 1, wc);
            if (!ok) break;
            float4* factors = reinterpret_cast<float4*>(smem + E::kFactorOff + n % E::kFactors * E::kFactorBytes);
            const uint32_t b4 = *reinterpret_cast<const uint32_t*>(smem + E::kKeyScaleOff + s * BN + lane * 4);
            factors[lane] =
                make_float4(__uint_as_float((b4 & 0xff) << 23) * p.key_bias, __uint_as_float((b4 & 0xff00) << 15) * p.key_bias,
                            __uint_as_float((b4 & 0xff0000) << 7) * p.key_bias, __uint_as_float(b4 >> 1 & 0x7f800000) * p.key_bias);
            __syncwarp();
            if (elect_one()) mbar_arrive(&bar.k_ready[s]);
            __syncwarp();
        }
    }
}

// The products P V of one-tile units, by a warp of its own: one that issues the scores' too comes to either late.
// Nothing orders the two but their barriers: scores, P and O have columns of their own.
template <int D, bool F16, int KERNEL, bool SMALL>
__device__ __forceinline__ void issue_values(const PagedDev& p, uint8_t* smem, Shared& bar) {
    using E = Cfg8<D, F16, 1, KERNEL, SMALL>;
    constexpr uint32_t kIdesc = idesc_h16(BM, D, false, true, F16);
    const WaitCtl wc{p.err, &bar.abort_flag, p.timeout_ns};
    const uint32_t tmem = __shfl_sync(kFull, bar.tmem_base, 0);
    Walk<1, KERNEL, kBytes> walk(p, bar);
    Unit w;
    uint32_t n = 0;
    bool ok = true;
    while (ok && walk.next(w)) {
        for (int j = 0; j < w.cnt_max && ok; ++j, ++n) {
            const uint32_t s = n % E::kWide, b = n & 1;
            ok = mbar_wait_warp(&bar.kv_full[s], (n / E::kWide) & 1, wc) && mbar_wait_warp(&bar.p_full[b], (n >> 1) & 1, wc);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                const uint64_t vd = vmajor_desc(smem_u32(smem + E::kWideOff + s * 2 * E::kTileBytes));
#pragma unroll
                for (int kk = 0; kk < BN / 16; ++kk)
                    mma_ts(tmem + E::kOCol, tmem + E::kPCol + b * 64 + kk * 8, vmajor_step(vd, kk), kIdesc, j > 0 || kk > 0 ? 1u : 0u);
                mma_commit(&bar.pv_done[b]);
                mma_commit(&bar.kv_empty[s]);
            }
            __syncwarp();
        }
    }
    if (elect_one()) {
        mma_commit(&bar.drain[1]);
        drain_wait(&bar.drain[1], 0, p.timeout_ns);
    }
    __syncwarp();
}

// The roles of kBytes but the softmax's.
template <int D, bool F16, int NT, int KERNEL, bool SMALL>
__device__ __forceinline__ void roles8(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const PagedDev& p, uint8_t* smem,
                                       Shared& bar) {
    using C = Cfg<D, NT, KERNEL, kBytes>;
    using E = Cfg8<D, F16, NT, KERNEL, SMALL>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const WaitCtl wc{p.err, &bar.abort_flag, p.timeout_ns};
    // Broadcast, so that the compiler knows what is the same in all lanes: an issuer's operands then stay in the registers
    // that its instructions take them from.
    const uint32_t tmem = __shfl_sync(kFull, bar.tmem_base, 0);
    Walk<NT, KERNEL, kBytes> walk(p, bar);
    Unit w;
    constexpr int kConvert = C::kProducer + 4;
    // Scores of tile t with the keys of stage s, into the columns from `to` on: the sum over Q's pieces.
    auto issue_s = [&](int t, uint32_t to, uint32_t s) {
        constexpr uint32_t kIdesc = ptx_f8::idesc_e4m3(BM, BN, false, false);
        const uint64_t kd = codes_desc<D>(smem_u32(smem + E::kKeyOff + s * E::kTileBytes));
#pragma unroll
        for (int piece = 0; piece < E::kPieces; ++piece) {
            const uint32_t idesc = piece > 0 ? kIdesc | 1u << 7 : kIdesc;  // A in E5M2
            const uint64_t qd = codes_desc<D>(smem_u32(smem + (t * E::kPieces + piece) * E::kTileBytes));
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk) {
                const uint32_t more = piece > 0 || kk > 0 ? 1u : 0u;
                if constexpr (E::kQTmem)
                    ptx_f8::mma_f8_ts(tmem + to, tmem + E::kQCol + piece * (D / 4) + kk * 8, step_desc(kd, kk * 2), idesc, more);
                else
                    ptx_f8::mma_f8_ss(tmem + to, step_desc(qd, kk * 2), step_desc(kd, kk * 2), idesc, more);
            }
        }
    };
    constexpr uint32_t kIdescO = idesc_h16(BM, D, false, true, F16);
    auto issue_pv = [&](uint32_t to, uint32_t from, uint32_t s, bool first) {
        const uint64_t vd = vmajor_desc(smem_u32(smem + E::kWideOff + s * 2 * E::kTileBytes));
#pragma unroll kIssueUnroll
        for (int kk = 0; kk < BN / 16; ++kk)
            mma_ts(tmem + to, tmem + from + kk * 8, vmajor_step(vd, kk), kIdescO, !first || kk > 0 ? 1u : 0u);
    };
    if (warp == C::kProducer || (C::kVProducer && warp == C::kFourth)) {
        // ------------------------------------------------ producers: as those of 16 bits, with a copy of scales a page
        const bool two = C::kVProducer;
        const int first = C::kVProducer && warp == C::kFourth ? 1 : 0;  // 0: K, 1: V
        const int end = two || first == 1 ? first + 1 : 2;
        const int box_rows = min(p.page_size, BN);
        const int my_key = lane * box_rows;
        uint32_t issued[2] = {0, 0};
        const uint32_t limit = p.stall_after > 0 ? (uint32_t)p.stall_after : UINT32_MAX;
        bool ok = true, bad = false;
        uint32_t n = 0;  // key tiles
        while (ok && (two || first == 0) && n < limit && walk.next(w)) {
            if (w.cnt_max == 0) continue;
            int page = 0;
            if (my_key < BN && w.k0 * BN + my_key < w.len) page = page_at(p, w.b, w.k0 * BN + my_key, &bad);
            w.cnt_max = min(w.cnt_max, (int)min(limit - n, (uint32_t)INT_MAX));
            for (int j = w.k0; j < w.k0 + w.cnt_max && ok; ++j, ++n) {
                const int key0 = j * BN;
                const bool active = my_key < BN && key0 + my_key < w.len;
                const uint32_t boxes = __popc(__ballot_sync(kFull, active));
                const int slot_row = (key0 + my_key) & (p.page_size - 1);
                const int my_page = page;
                if (j + 1 < w.k0 + w.cnt_max && my_key < BN && key0 + BN + my_key < w.len)
                    page = page_at(p, w.b, key0 + BN + my_key, &bad);
                // a page that the cache does not have reads as zeros, whatever the scales
                const long long at_page = my_page < p.num_pages ? my_page : 0;
                for (int kv = first; kv < end; ++kv) {
                    const uint32_t s = n % (kv == 0 ? E::kKeys : E::kValues), use = n / (kv == 0 ? E::kKeys : E::kValues);
                    uint64_t* full = kv == 0 ? &bar.k_full[s] : &bar.v_full[s];
                    ok = mbar_wait_warp(kv == 0 ? &bar.k_empty[s] : &bar.v_empty[s], (use & 1) ^ 1, wc);
                    if (!ok) break;
                    if (elect_one()) mbar_arrive_expect_tx(full, boxes * (uint32_t)(box_rows * (D + 1)));
                    __syncwarp();
                    if (active) {
                        uint8_t* dst = smem + (kv == 0 ? E::kKeyOff : E::kValueOff) + s * E::kTileBytes + my_key * D;
                        uint8_t* scales = smem + (kv == 0 ? E::kKeyScaleOff : E::kValueScaleOff) + s * BN + my_key;
                        const uint8_t* src = kv == 0 ? p.k_scale + at_page * p.ks_page + w.h * p.ks_head
                                                     : p.v_scale + at_page * p.vs_page + w.h * p.vs_head;
                        tma_load_4d(dst, kv == 0 ? &tm_k : &tm_v, full, 0, slot_row, w.h, my_page);
                        bulk_load(scales, src + slot_row, (uint32_t)box_rows, full);
                    }
                    __syncwarp();
                    issued[kv] = n + 1;
                }
            }
        }
        if (bad) atomicCAS(p.err, 0, ATTN_ERR_INVALID);
        if (lane == 0) {
            if (first == 0) bar.issued[0] = issued[0];
            if (end == 2 && (two || first == 0)) bar.issued[1] = issued[1];
        }
    } else if (warp == C::kTail) {
        // ------------------------------------------------ the CTA's slots, and Q of small units
        uint32_t units = 0;
        bool ok = true;
        int4 slot0 = make_int4(kNone, 0, 0, 0), slot1 = slot0;
        while (walk.next(w)) {
            if (!(w.first && w.last)) {
                const int4 m = make_int4(w.last ? kLast : kPart, w.row0, w.ntok, w.h);
                if (w.first)
                    slot1 = m;
                else
                    slot0 = m;
            }
            if (!SMALL || w.cnt_max == 0 || !ok) continue;  // the slots are written whatever happens
            const uint32_t at = units % E::kQSlots;
            ok = mbar_wait_warp(&bar.q_empty[1 + at], ((units / E::kQSlots) & 1) ^ 1, wc);
            if (!ok) continue;
            split_unit<D, F16, E::kQPitch>(p, w, smem + E::kQSlotOff + at * E::kQSlot, lane);
            __syncwarp();
            if (elect_one()) mbar_arrive(&bar.q_full[1 + at]);
            __syncwarp();
            ++units;
        }
        if (lane < 2) p.meta[blockIdx.x * 2 + lane] = lane == 0 ? slot0 : slot1;
    } else if (warp >= kConvert) {
        // ------------------------------------------------ converters: the keys' factors, the values in 16 bits
        // All on every tile, in order: a wait tells the phases of a stage apart only while no use of it is passed
        // over, and none can pass while the wait stands.
        constexpr int W = E::kMakers;
        const int c = warp - kConvert;
        if constexpr (NT == 1 && KERNEL == kOne) {
            if (c == W) make_factors<D, F16, KERNEL, SMALL>(p, smem, bar);
            if (c == W + 1) issue_values<D, F16, KERNEL, SMALL>(p, smem, bar);
        }
        uint32_t n = 0;
        bool ok = c < W;
        while (ok && walk.next(w)) {
            for (int j = 0; j < w.cnt_max && ok; ++j, ++n) {
                const uint32_t sk = n % E::kKeys, sv = n % E::kValues, so = n % E::kWide;
                const uint32_t pk = (n / E::kKeys) & 1, pv = (n / E::kValues) & 1, po = ((n / E::kWide) & 1) ^ 1;
                const unsigned ready = look(&bar.k_full[sk], pk, &bar.v_full[sv], pv, &bar.kv_empty[so], po, &bar.k_full[sk], pk);
                if constexpr (NT == 2) {
                    ok = (ready & 1) || mbar_wait_warp(&bar.k_full[sk], pk, wc);
                    if (!ok) break;
                    const int at = c * 32 + lane;
                    reinterpret_cast<float*>(smem + E::kFactorOff)[n % E::kFactors * BN + at] =
                        __uint_as_float((uint32_t)smem[E::kKeyScaleOff + sk * BN + at] << 23) * p.key_bias;
                    __syncwarp();
                    if (elect_one()) mbar_arrive(&bar.k_ready[sk]);
                }
                ok = ((ready & 2) || mbar_wait_warp(&bar.v_full[sv], pv, wc)) &&
                     ((ready & 4) || mbar_wait_warp(&bar.kv_empty[so], po, wc));
                if (!ok) break;
                widen_tile<D, F16, W, KERNEL == kMixed>(smem + E::kValueOff + sv * E::kTileBytes, smem + E::kValueScaleOff + sv * BN,
                                      smem + E::kWideOff + so * 2 * E::kTileBytes, w.len - (w.k0 + j) * BN, c, lane);
                fence_proxy_async_smem();
                __syncwarp();
                if (elect_one()) {
                    mbar_arrive(&bar.kv_full[so]);
                    mbar_arrive(&bar.v_empty[sv]);
                }
                __syncwarp();
            }
        }
    } else if (NT == 1 && warp == C::kIssuer) {
        // ------------------------------------------------ issuer of one tile's scores
        uint32_t n = 0, units = 0;
        bool ok = true;
        while (ok && walk.next(w)) {
            if (w.cnt_max == 0) continue;
            ok = mbar_wait_warp(&bar.q_full[0], units++ & 1, wc);
            for (int j = 0; j < w.cnt_max && ok; ++j, ++n) {
                const uint32_t s = n % E::kKeys;
                ok = mbar_wait_warp(&bar.k_ready[s], (n / E::kKeys) & 1, wc) && mbar_wait_warp(&bar.s_free[0], (n & 1) ^ 1, wc);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    issue_s(0, 0, s);
                    mma_commit(&bar.s_full[0]);
                    mma_commit(&bar.k_empty[s]);
                }
                __syncwarp();
            }
        }
        if (elect_one()) {
            mma_commit(&bar.drain[0]);
            drain_wait(&bar.drain[0], 0, p.timeout_ns);
        }
        __syncwarp();
    } else if (NT == 2 && !C::kOneIssuer && (warp == C::kIssuer || warp == C::kFourth)) {
        // ------------------------------------------------ issuers, one per query tile: as those of 16 bits with P in
        // columns of its own
        const int t = warp == C::kIssuer ? 0 : 1;
        uint32_t n = 0, n_s = 0, n_p = 0, units = 0;
        bool ok = true;
        while (ok && walk.next(w)) {
            if (w.cnt_max == 0) continue;
            const int cnt = w.cnt(t);
            if (cnt > 0) {
                ok = mbar_wait_warp(&bar.q_full[t], units++ & 1, wc);
                if (!ok) break;
                tc_fence_after();
            }
            for (int j = 0; j <= w.cnt_max && ok; ++j) {
                const uint32_t sK = n % E::kKeys, sV = (n + E::kWide - 1) % E::kWide;  // V of the tile before
                const uint32_t k_phase = (n / E::kKeys) & 1, v_phase = ((n - 1) / E::kWide) & 1;
                const unsigned ready = look(&bar.k_ready[sK], k_phase, &bar.s_free[t], (n_s - 1) & 1, &bar.kv_full[sV], v_phase,
                                            &bar.p_full[t], n_p & 1);
                if (j < w.cnt_max) {
                    ok = (ready & 1) || mbar_wait_warp(&bar.k_ready[sK], k_phase, wc);
                    if (ok && j < cnt && n_s > 0) ok = (ready & 2) || mbar_wait_warp(&bar.s_free[t], (n_s - 1) & 1, wc);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        if (j < cnt) {
                            issue_s(t, t * BN, sK);
                            mma_commit(&bar.s_full[t]);
                        }
                        mma_commit(&bar.k_empty[sK]);
                    }
                    __syncwarp();
                    if (j < cnt) ++n_s;
                }
                if (j > 0) {
                    ok = (ready & 4) || mbar_wait_warp(&bar.kv_full[sV], v_phase, wc);
                    if (ok && j <= cnt) {
                        ok = (ready & 8) || mbar_wait_warp(&bar.p_full[t], n_p & 1, wc);
                        ++n_p;
                    }
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        if (j <= cnt) {
                            issue_pv(C::o_col(t), C::p_col(t), sV, j == 1);
                            mma_commit(&bar.pv_done[t]);
                        }
                        mma_commit(&bar.kv_empty[sV]);
                    }
                    __syncwarp();
                }
                if (j < w.cnt_max) ++n;
            }
        }
        if (elect_one()) {
            mma_commit(&bar.drain[t]);
            drain_wait(&bar.drain[t], 0, p.timeout_ns);
        }
        __syncwarp();
    } else if (NT == 2 && C::kOneIssuer && warp == C::kIssuer) {
        // ------------------------------------------------ the one issuer of two tiles with P over S: as that of 16 bits
        uint32_t n = 0, pcnt0 = 0, pcnt1 = 0, units0 = 0, units1 = 0;
        bool ok = true;
        while (ok && walk.next(w)) {
            if (w.cnt_max == 0) continue;
            uint32_t sK = n % E::kKeys;
            ok = mbar_wait_warp(&bar.k_ready[sK], (n / E::kKeys) & 1, wc);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (!ok || w.cnt(t) == 0) continue;
                uint32_t& units = t == 0 ? units0 : units1;
                ok = mbar_wait_warp(&bar.q_full[t], units++ & 1, wc);
                tc_fence_after();
                if (ok && elect_one()) {
                    issue_s(t, t * BN, sK);
                    mma_commit(&bar.s_full[t]);
                }
                __syncwarp();
            }
            if (!ok) break;
            for (int j = 1; j <= w.cnt_max && ok; ++j) {
                const uint32_t sV = n % E::kWide, v_phase = (n / E::kWide) & 1;  // V of tile j - 1
                if (elect_one()) {
                    if (j > 1) mma_commit(&bar.kv_empty[(n + E::kWide - 1) % E::kWide]);
                    mma_commit(&bar.k_empty[sK]);
                }
                __syncwarp();
                ++n;
                sK = n % E::kKeys;
                const uint32_t k_phase = (n / E::kKeys) & 1;
                const unsigned ready = look(&bar.k_ready[sK], k_phase, &bar.kv_full[sV], v_phase, &bar.p_full[0], pcnt0 & 1,
                                            &bar.p_full[1], pcnt1 & 1);
                if (j < w.cnt_max) {
                    ok = (ready & 1) || mbar_wait_warp(&bar.k_ready[sK], k_phase, wc);
                    if (!ok) break;
                }
                ok = (ready & 2) || mbar_wait_warp(&bar.kv_full[sV], v_phase, wc);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    if (!ok || j > w.cnt(t)) continue;
                    uint32_t& pcnt = t == 0 ? pcnt0 : pcnt1;
                    ok = (ready & (t == 0 ? 4 : 8)) || mbar_wait_warp(&bar.p_full[t], pcnt & 1, wc);
                    if (!ok) continue;
                    ++pcnt;
                    tc_fence_after();
                    if (elect_one()) {
                        issue_pv(C::o_col(t), C::p_col(t), sV, j == 1);
                        if (j == w.cnt(t)) mma_commit(&bar.o_full[t]);  // last product of this tile
                        if (j < w.cnt(t)) {
                            issue_s(t, t * BN, sK);
                            mma_commit(&bar.s_full[t]);
                        }
                    }
                    __syncwarp();
                }
            }
            if (!ok) break;
            if (elect_one()) mma_commit(&bar.kv_empty[(n + E::kWide - 1) % E::kWide]);  // the last V
            __syncwarp();
        }
        if (elect_one()) {
            mma_commit(&bar.drain[0]);
            drain_wait(&bar.drain[0], 0, p.timeout_ns);
        }
        __syncwarp();
    }
}

// Writes what a thread has of its row r of tile t at a unit's end: O and LSE of a whole unit, or the part's state.
// All lanes of a warp.
template <int D, bool F16, int TILES>
__device__ __forceinline__ void finish_row(const PagedDev& p, const int4& u, int t, int r, int my_tok, int my_head, int rows, int cnt,
                                           uint32_t tO, float m_ref, float m_row, float l) {
    const bool held = r < rows && my_tok < u.y, first = u.w & 1, last = u.w & 2;
    const float den = o_divisor<F16>(l, m_row, m_ref);
    if (first && last) {
        const float inv = den > 0.f ? 1.f / den : 0.f;
        // a row without keys is 0, though its products of 0 and a value may be NaN
        const uint32_t keep = l == 0.f ? 0u : ~0u;
        const long long row = u.x + my_tok, head = u.z * p.G + my_head;
        uint16_t* orow = reinterpret_cast<uint16_t*>(p.o) + row * p.o_sr + head * p.o_sh;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 64) {
            uint32_t ov[64];
            if (cnt > 0) {
                tmem_ld32_at<0>(tO + c0, ov);
                tmem_ld32_at<32>(tO + c0 + 32, ov);
                tmem_wait_ld();
            } else {
#pragma unroll
                for (int i = 0; i < 64; ++i) ov[i] = 0;
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float2 x = fmul2(make_float2(__uint_as_float(ov[2 * i]), __uint_as_float(ov[2 * i + 1])),
                                       make_float2(inv, inv));
                ov[i] = pack_h16<F16>(x.x, x.y) & keep;
            }
            if (held) {
                if (p.o_wide) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) store32(orow + c0 + 16 * q, &ov[8 * q]);
                } else {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        *reinterpret_cast<uint4*>(orow + c0 + 8 * q) =
                            make_uint4(ov[4 * q], ov[4 * q + 1], ov[4 * q + 2], ov[4 * q + 3]);
                }
            }
        }
        if (held) p.lse[head * p.T + row] = row_lse(m_ref, l);
    } else {
        // the part's state of this row; a row without keys in it is m = -inf, and its o is not read. NaN
        // scores leave m_ref at -inf and l NaN: such a row has keys, and its m is any other number.
        float4* rec = record(p.part, blockIdx.x * 2 + (first ? 1 : 0), TILES, t, rows, D);
        if (held) rec[r] = make_float4(l == 0.f ? -INFINITY : fmaxf(m_ref, -FLT_MAX), l, den, 0.f);
        if (cnt > 0) {
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
                uint32_t ov[32];
                tmem_ld32(tO + c0, ov);
                tmem_wait_ld();
                if (held) {
                    float4* dst = rec + (1 + c0 / 4) * rows + r;
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        dst[q * rows] = make_float4(__uint_as_float(ov[4 * q]), __uint_as_float(ov[4 * q + 1]),
                                                    __uint_as_float(ov[4 * q + 2]), __uint_as_float(ov[4 * q + 3]));
                }
            }
        }
    }
}

// The softmax of units of one tile.
//
// A thread has a row, but in small units a row has a lane of tensor memory in each of the four warps: every warp has a
// copy of Q's rows, so S too, and takes 32 of a tile's 128 keys. The copies' P are 0 at the other keys, so that their O
// add up to the row's, each with a running maximum of its own; they are merged at the unit's end like the parts of a
// unit that was cut (64 sequences of 8192 keys 314 us with a row in one thread, 160 with copies; 512 of 128 keys 158 and 143, one
// of 517 keys 17 to 19 either way).
template <int D, bool F16, int KERNEL, bool SMALL>
__device__ __forceinline__ void softmax_one(const PagedDev& p, uint8_t* smem, Shared& bar) {
    using C = Cfg<D, 1, KERNEL, kBytes>;
    using E = Cfg8<D, F16, 1, KERNEL, SMALL>;
    constexpr bool kCopies = SMALL;
    constexpr int COLS = SMALL ? 32 : 128;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const WaitCtl wc{p.err, &bar.abort_flag, p.timeout_ns};
    const int rows = p.tok_tile * p.G;
    const int r = kCopies ? lane : threadIdx.x;
    const int my_tok = r / p.G, my_head = r % p.G, col0 = kCopies ? warp * 32 : 0;
    const uint32_t tmem = bar.tmem_base + ((uint32_t)(warp * 32) << 16);
    const uint32_t tO = tmem + E::kOCol, tP = tmem + E::kPCol;
    uint32_t scnt = 0, mcnt = 0, units = 0;  // scnt: tiles before this one
    bool ok = true;
    if constexpr (kCopies) {  // P at the other copies' keys
        uint32_t zero[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) zero[i] = 0;
#pragma unroll
        for (int c = 0; c < 128; c += 32) tmem_st32(tP + c, zero);
        tmem_wait_st();
    }
    Walk<1, KERNEL, kBytes> walk(p, bar);
    Unit w;
    bool more = walk.next(w);
    float row_c = p.c;
    int factors = 0;
    auto take_q = [&]() {
        if constexpr (kCopies) {
            const uint32_t at = units % E::kQSlots;
            ok = mbar_wait_warp(&bar.q_full[1 + at], (units / E::kQSlots) & 1, wc);
            ++units;
            const uint8_t* slot = smem + E::kQSlotOff + at * E::kQSlot;
            // lanes without a row have whatever lies there; they must not move a maximum
            const float f = lane < rows && my_tok < w.ntok ? reinterpret_cast<const float*>(slot + 32 * E::kPieces * E::kQPitch)[lane] : 0.f;
            row_c = row_factor(p.c, f);
#pragma unroll
            for (int k = 0; k < E::kPieces; ++k)
#pragma unroll
                for (int c = 0; c < D; c += 64) {
                    uint32_t x[16];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 v = *reinterpret_cast<const uint4*>(slot + (k * 32 + lane) * E::kQPitch + c + i * 16);
                        x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
                    }
                    tmem_st16(tmem + E::kQCol + (k * D + c) / 4, x);
                }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (elect_one()) mbar_arrive(&bar.q_empty[1 + at]);
            __syncwarp();
        } else {
            const uint16_t* src = nullptr;
            if (r < rows && my_tok < w.ntok) src = p.q + (w.row0 + my_tok) * p.q_sr + (w.h * p.G + my_head) * p.q_sh;
            __syncwarp();
            row_c = row_factor(p.c, split_row<D, F16, true>(src, tmem + E::kQCol, nullptr, r));
        }
        mbar_arrive(&bar.q_full[0]);
    };
    if (more && w.cnt0 > 0) take_q();
    while (ok && more) {
        const int4 u = make_int4(w.row0, w.ntok, w.h, (w.first ? 1 : 0) + (w.last ? 2 : 0));
        const int cnt = w.cnt0, k0 = w.k0;
        const int lim = w.causal ? min(w.len, w.base + my_tok + 1) : w.len;
        const int lim_first = w.causal ? min(w.len, w.base + 1) : w.len;
        const int ctx = !w.causal && p.tree != nullptr ? w.ctx : INT_MAX;
        float m_ref = -INFINITY, m_row = -INFINITY, l = 0.f;
        bool s_ready = false;
        for (int j = 0; j < cnt; ++j) {
            const uint32_t b = scnt & 1;
            ok = s_ready || mbar_wait(&bar.s_full[0], scnt & 1, wc);
            ok = __all_sync(kFull, ok);
            if (!ok) break;
            tc_fence_after();
            uint32_t su[COLS];
            tmem_ld32_at<0>(tmem + col0, su);
            if constexpr (!kCopies) {
                tmem_ld32_at<32>(tmem + 32, su);
                tmem_ld32_at<64>(tmem + 64, su);
                tmem_ld32_at<96>(tmem + 96, su);
            }
            const float4* f = reinterpret_cast<const float4*>(smem + E::kFactorOff + factors * E::kFactorBytes) + col0 / 4;
            float4 f4[8];
            if constexpr (SMALL) {  // beside the scores
#pragma unroll
                for (int i = 0; i < 8; ++i) f4[i] = f[i];
            }
            tmem_wait_ld();
            tc_fence_before();
            mbar_arrive(&bar.s_free[0]);  // the scores are in registers
#pragma unroll
            for (int i = 0; i < COLS / 4; ++i) {
                const float4 x = SMALL ? f4[i % 8] : f[i];
                const float2 a = fmul2(make_float2(__uint_as_float(su[4 * i]), __uint_as_float(su[4 * i + 1])), make_float2(x.x, x.y));
                const float2 c = fmul2(make_float2(__uint_as_float(su[4 * i + 2]), __uint_as_float(su[4 * i + 3])), make_float2(x.z, x.w));
                su[4 * i] = __float_as_uint(a.x), su[4 * i + 1] = __float_as_uint(a.y);
                su[4 * i + 2] = __float_as_uint(c.x), su[4 * i + 3] = __float_as_uint(c.y);
            }
            factors = factors + 1 == E::kFactors ? 0 : factors + 1;
            const int key0 = (k0 + j) * BN + col0;
            if (key0 > ctx - COLS) {
                uint32_t bits[COLS / 32];
                tree_bits(p, r < rows && my_tok < w.ntok ? p.tree + (w.row0 + my_tok) * p.tree_stride : nullptr, key0, ctx, w.len,
                          bits);
#pragma unroll
                for (int col = 0; col < COLS; ++col)
                    if (!(bits[col / 32] >> (col & 31) & 1)) su[col] = __float_as_uint(-INFINITY);
            } else if (key0 + COLS > lim_first) {
                const int out = lim - key0;
#pragma unroll
                for (int col = 0; col < COLS; ++col)
                    if (col >= out) su[col] = __float_as_uint(-INFINITY);
            }
            float mx[COLS / 16];
#pragma unroll
            for (int c = 0; c < COLS / 16; ++c) {
                mx[c] = fmaxf(__uint_as_float(su[16 * c]), __uint_as_float(su[16 * c + 1]));
#pragma unroll
                for (int e = 2; e < 16; e += 2)
                    mx[c] = fmax3(mx[c], __uint_as_float(su[16 * c + e]), __uint_as_float(su[16 * c + e + 1]));
            }
            float m_tile = mx[0];
#pragma unroll
            for (int c = 1; c < COLS / 16; ++c) m_tile = fmaxf(m_tile, mx[c]);
            m_tile *= row_c;
            m_row = fmaxf(m_row, m_tile);
            float m_new = m_ref;
            if (m_tile > m_ref + kRescaleThreshold) m_new = m_tile;
            const bool moved = m_new != m_ref;
            const float alpha = moved ? ex2(m_ref - m_new) : 1.f;  // 0 when m_ref = -inf
            const bool rescale = j > 0 && __any_sync(kFull, moved && m_ref != -INFINITY);
            m_ref = m_new;
            const float neg_m = (m_ref == -INFINITY) ? 0.f : -m_ref;
            const float2 cc2 = make_float2(row_c, row_c), nm2 = make_float2(neg_m, neg_m);
            float2 suma = make_float2(0.f, 0.f), sumb = make_float2(0.f, 0.f);
            // The product of the tile before the last has read this P: looked at beside other work.
            const bool p_free = scnt < 2 || mbar_test(&bar.pv_done[b], ((scnt >> 1) & 1) ^ 1);
#pragma unroll
            for (int i = 0; i < COLS / 2; ++i) {
                const float2 x = ffma2(make_float2(__uint_as_float(su[2 * i]), __uint_as_float(su[2 * i + 1])), cc2, nm2);
                const float2 pp = make_float2(ex2(x.x), ex2(x.y));
                float2& sum = i & 1 ? sumb : suma;
                sum = fadd2(sum, pp);
                su[i] = pack_h16<F16>(pp.x, pp.y);
            }
            ok = p_free || mbar_wait(&bar.pv_done[b], ((scnt >> 1) & 1) ^ 1, wc);
            ok = __all_sync(kFull, ok);
            if (!ok) break;
            if (rescale) {  // the tile before has written O
                ok = mbar_wait(&bar.pv_done[b ^ 1], ((scnt - 1) >> 1) & 1, wc);
                ok = __all_sync(kFull, ok);
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t ov[32];
                    tmem_ld32(tO + c0, ov);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
                    tmem_st32(tO + c0, ov);
                }
            }
            tc_fence_after();
            if constexpr (kCopies) {
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) pk[i] = su[i];
                tmem_st16(tP + b * 64 + warp * 16, pk);
            } else {
                tmem_st32_at<0>(tP + b * 64, su);
                tmem_st32_at<32>(tP + b * 64 + 32, su);
            }
            ++scnt;
            s_ready = j + 1 < cnt && mbar_test(&bar.s_full[0], scnt & 1);
            l = l * alpha + ((suma.x + suma.y) + (sumb.x + sumb.y));
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&bar.p_full[b]);
        }
        if (!ok) break;
        more = walk.next(w);  // while the last product runs
        if (more && w.cnt0 > 0) take_q();  // every product with this unit's has been waited for
        if (!ok) break;
        const bool first = u.w & 1, last = u.w & 2;
        if (cnt > 0) {
            ok = mbar_wait(&bar.pv_done[(scnt - 1) & 1], ((scnt - 1) >> 1) & 1, wc);
            ok = __all_sync(kFull, ok);
            if (!ok) break;
            tc_fence_after();
        }
        if constexpr (!kCopies) {
            finish_row<D, F16, C::Kernel::kTiles>(p, u, 0, r, my_tok, my_head, rows, cnt, tO, m_ref, m_row, l);
            tc_fence_before();
            continue;
        }
        // Merging, rows and columns in rounds that the area holds: `span` rows of `cols` columns, a thread 8 columns of row rr.
        const int span = bar.most_rows <= 8 ? 8 : bar.most_rows <= 16 ? 16 : 32;
        const int most = 32 * 32 / span, cols = min(D, most), pitch = most + 4;
        float4* states = reinterpret_cast<float4*>(smem + E::kStateOff);
        float* area = reinterpret_cast<float*>(smem + E::kMergeOff);
        auto meet = [&]() {
            mbar_arrive(&bar.merged);
            ok = __all_sync(kFull, mbar_wait(&bar.merged, mcnt & 1, wc));
            ++mcnt;
        };
        // The copy's state, as that of a part of a unit. Every warp is done with the unit before, or there would be no P for
        // the products above.
        if (cnt > 0 && lane < span)
            states[warp * span + lane] =
                make_float4(l == 0.f ? -INFINITY : fmaxf(m_ref, -FLT_MAX), l, o_divisor<F16>(l, m_row, m_ref), 0.f);
        const int rr = threadIdx.x % span, group = threadIdx.x / span, tok = rr / p.G;
        const bool held = rr < rows && tok < u.y && group * 8 < cols;
        const long long row = u.x + tok, head = u.z * p.G + rr % p.G;
        uint16_t* orow = reinterpret_cast<uint16_t*>(p.o) + row * p.o_sr + head * p.o_sh;
        float4* rec = record(p.part, blockIdx.x * 2 + (first ? 1 : 0), C::Kernel::kTiles, 0, rows, D) + rr;
#pragma unroll 1
        for (int c0 = 0; c0 < D && ok; c0 += cols) {
            if (cnt > 0) {
                if (c0 > 0) meet();  // the area has been read
#pragma unroll 1
                for (int c1 = 0; c1 < cols && ok; c1 += 32) {
                    uint32_t ov[32];
                    tmem_ld32(tO + c0 + c1, ov);
                    tmem_wait_ld();
                    if (lane < span) {
                        float4* dst = reinterpret_cast<float4*>(area + (warp * span + lane) * pitch + c1);
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            dst[q] = make_float4(__uint_as_float(ov[4 * q]), __uint_as_float(ov[4 * q + 1]),
                                                 __uint_as_float(ov[4 * q + 2]), __uint_as_float(ov[4 * q + 3]));
                    }
                }
                tc_fence_before();
                meet();
                if (!ok) break;
            }
            float m = -INFINITY, sum = 0.f, den = 0.f, out[8];
            float4 st[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                st[k] = cnt > 0 ? states[k * span + rr] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
                m = fmaxf(m, st[k].x);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) out[i] = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (st[k].x == -INFINITY) continue;  // no key of this row in the copy
                const float f = ex2(st[k].x - m);
                sum = fmaf(f, st[k].y, sum);
                den = fmaf(f, st[k].z, den);
                const float4* src = reinterpret_cast<const float4*>(area + (k * span + rr) * pitch + group * 8);
                const float4 a = src[0], c = src[1];
                out[0] = fmaf(f, a.x, out[0]), out[1] = fmaf(f, a.y, out[1]), out[2] = fmaf(f, a.z, out[2]);
                out[3] = fmaf(f, a.w, out[3]), out[4] = fmaf(f, c.x, out[4]), out[5] = fmaf(f, c.y, out[5]);
                out[6] = fmaf(f, c.z, out[6]), out[7] = fmaf(f, c.w, out[7]);
            }
            if (!held) continue;
            if (first && last) {
                const float inv = den > 0.f ? 1.f / den : 0.f;
                *reinterpret_cast<uint4*>(orow + c0 + group * 8) =
                    make_uint4(pack_h16<F16>(out[0] * inv, out[1] * inv), pack_h16<F16>(out[2] * inv, out[3] * inv),
                               pack_h16<F16>(out[4] * inv, out[5] * inv), pack_h16<F16>(out[6] * inv, out[7] * inv));
                if (c0 == 0 && group == 0) p.lse[head * p.T + row] = row_lse(m, sum);
            } else {
                if (c0 == 0 && group == 0) rec[0] = make_float4(m, sum, den, 0.f);
                const int g4 = (c0 + group * 8) / 4;
                rec[(1 + g4) * rows] = make_float4(out[0], out[1], out[2], out[3]);
                rec[(2 + g4) * rows] = make_float4(out[4], out[5], out[6], out[7]);
            }
        }
    }
}

// The work of a CTA on units of NT tiles, from the located piece of the line to its end.
template <int D, bool F16, int NT, int KERNEL, int VAR>
__device__ __forceinline__ void work(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                     const PagedDev& p, uint8_t* smem, Shared& bar) {
    using C = Cfg<D, NT, KERNEL, VAR>;
    constexpr uint32_t kIdescS = idesc_h16(BM, BN, false, false, F16);
    constexpr uint32_t kIdescO = idesc_h16(BM, D, false, true, F16);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const WaitCtl wc{p.err, &bar.abort_flag, p.timeout_ns};
    const bool copies = VAR == kBytes && NT == 1 && bar.sm_warps == 1;
    if (threadIdx.x == 0) {
        const uint32_t rows = copies ? 128u : 32u * (uint32_t)bar.sm_warps;  // softmax threads of a tile
        for (int i = 0; i < 4; ++i) {
            const bool slot = VAR == kBytes && NT == 1 && i > 0;  // of small units' pieces
            mbar_init(&bar.q_full[i], VAR == kBytes && !slot ? rows : 1);
            mbar_init(&bar.q_empty[i], slot ? 4 : 1);
        }
        if constexpr (VAR == kBytes) {
            using E = Cfg8<D, F16, NT, KERNEL, false>;
            constexpr uint32_t kConverters = E::kMakers;
            for (int s = 0; s < 8; ++s) {
                mbar_init(&bar.k_full[s], 1);
                mbar_init(&bar.k_ready[s], NT == 1 ? 1 : kConverters);
                mbar_init(&bar.k_empty[s], C::kIssuers);
                mbar_init(&bar.v_full[s], 1);
                mbar_init(&bar.v_empty[s], kConverters);
            }
            for (int s = 0; s < E::kWide; ++s) {
                mbar_init(&bar.kv_full[s], kConverters);
                mbar_init(&bar.kv_empty[s], C::kIssuers);
            }
        } else {
            for (int s = 0; s < C::kStages; ++s) {
                mbar_init(&bar.kv_full[s], 1);
                mbar_init(&bar.kv_empty[s], C::kIssuers);
                mbar_init(&bar.v_tail[s], 1);
            }
        }
        for (int t = 0; t < (VAR == kBytes ? 2 : NT); ++t) {
            mbar_init(&bar.s_full[t], 1);
            mbar_init(&bar.p_full[t], rows);
            mbar_init(&bar.o_full[t], 1);
            mbar_init(&bar.s_free[t], rows);
            mbar_init(&bar.pv_done[t], 1);
            mbar_init(&bar.drain[t], 1);
        }
        if (VAR == kBytes) mbar_init(&bar.merged, 128);
        fence_mbar_init();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem_base;
    const uint32_t sQ = smem_u32(smem + C::kQOff);
    const uint32_t sKV = smem_u32(smem + C::kKVOff);
    // One tile: a product reads 128 rows from a slot's start; what lies behind the tile's own rows only reaches
    // rows that nobody reads.
    const uint32_t q_half = NT == 1 ? (uint32_t)((p.tok_tile * p.G + 7) / 8 * 1024) : BM * 128;  // bytes of a box
    const uint32_t q_stride = q_half * C::kBoxes;
    const uint32_t q_slots = NT == 1 ? min(4u, (uint32_t)C::kQBytes / q_stride) : C::kQTiles;

    if (warp >= C::kProducer) {
        if constexpr (C::Kernel::kRebalance) regs_decrease<C::Kernel::kOtherRegs>();
        if constexpr (VAR == kBytes) {
            if (NT == 1 && copies)
                roles8<D, F16, NT, KERNEL, NT == 1>(tm_k, tm_v, p, smem, bar);
            else
                roles8<D, F16, NT, KERNEL, false>(tm_k, tm_v, p, smem, bar);
        } else {
        Walk<NT, KERNEL, VAR> walk(p, bar);
        Unit w;
        if (warp == C::kProducer || (C::kVProducer && warp == C::kFourth)) {
            // ------------------------------------------------ K and V producers
            // Small pages make many small copies, which one warp issues at about one in 90 cycles: K and V are
            // issued by a warp each where there is one for V (64 sequences of 8192 keys in 16-token pages 275 us,
            // 335 by one warp; in 64-token pages 244 by two, 239 by one).
            const bool two = C::kVProducer && p.page_size < 64;
            const int first = C::kVProducer && warp == C::kFourth ? 1 : 0;  // 0: K, 1: V
            const int end = two || first == 1 ? first + 1 : 2;
            const int box_rows = min(p.page_size, BN);   // keys a box holds
            const uint32_t box_bytes = (uint32_t)box_rows * 128;
            const int my_key = lane * box_rows;          // of a tile, where this lane has a box
            uint32_t it = 0;                             // ring items: K and V in turn
            const uint32_t limit = p.stall_after > 0 ? 2u * (uint32_t)p.stall_after : UINT32_MAX;
            bool ok = true, bad = false;
            while (ok && (two || first == 0) && it < limit && walk.next(w)) {
                if (w.cnt_max == 0) continue;
                int page = 0;  // this lane's page of the current tile
                if (my_key < BN && w.k0 * BN + my_key < w.len) page = page_at(p, w.b, w.k0 * BN + my_key, &bad);
                w.cnt_max = min(w.cnt_max, (int)((limit - it) / 2));
                for (int j = w.k0; j < w.k0 + w.cnt_max && ok; ++j, it += 2) {
                    const int key0 = j * BN;
                    const bool active = my_key < BN && key0 + my_key < w.len;
                    const uint32_t boxes = __popc(__ballot_sync(kFull, active));
                    const int slot_row = (key0 + my_key) & (p.page_size - 1);
                    const int my_page = page;
                    // the next tile's page, looked up while this one's copies are issued
                    if (j + 1 < w.k0 + w.cnt_max && my_key < BN && key0 + BN + my_key < w.len)
                        page = page_at(p, w.b, key0 + BN + my_key, &bad);
                    const bool tail = key0 + BN > w.len;
                    for (int kv = first; kv < end; ++kv) {
                        const uint32_t s = (it + kv) % C::kStages;
                        ok = mbar_wait_warp(&bar.kv_empty[s], (((it + kv) / C::kStages) & 1) ^ 1, wc);
                        if (!ok) {
                            it += kv - 2;  // ends as the first item not issued here
                            break;
                        }
                        uint64_t* full = kv == 1 && tail ? &bar.v_tail[s] : &bar.kv_full[s];
                        if (elect_one()) mbar_arrive_expect_tx(full, boxes * box_bytes * C::kBoxes);
                        __syncwarp();
                        if (active) {
                            uint8_t* dst = smem + C::kKVOff + s * C::kTileBytes + my_key * 128;
                            for (int bx = 0; bx < C::kBoxes; ++bx)
                                tma_load_4d(dst + bx * BN * 128, kv == 0 ? &tm_k : &tm_v, full, bx * 64, slot_row, w.h,
                                            my_page);
                        }
                        __syncwarp();
                    }
                }
            }
            if (bad) atomicCAS(p.err, 0, ATTN_ERR_INVALID);
            if (lane == 0 && (two || first == 0)) {
                bar.issued[first] = it;
                if (!two) bar.issued[1] = it;
            }
        } else if (warp == C::kTail) {
            // ------------------------------------------------ Q, rows of V beyond the sequence, the CTA's slots
            const uint32_t q_bytes = (uint32_t)(p.tok_tile * p.G) * 128 * C::kBoxes;
            uint32_t it = 0, phases = 0;          // ring items; phase of v_tail[s] in bit s
            uint32_t q_at = 0, q_used = 0;        // slot of the next Q tile; uses of each slot, 8 bits a slot
            int4 slot0 = make_int4(kNone, 0, 0, 0), slot1 = slot0;
            bool ok = true;
            while (walk.next(w)) {
                if (!(w.first && w.last)) {
                    const int4 m = make_int4(w.last ? kLast : kPart, w.row0, w.ntok, w.h);
                    if (w.first)
                        slot1 = m;
                    else
                        slot0 = m;
                }
                if (w.cnt_max == 0 || !ok) continue;  // the slots are written whatever happens
#pragma unroll 1
                for (int t = 0; t < NT && ok; ++t) {
                    if (w.cnt(t) == 0) continue;
                    const uint32_t i = q_at;
                    ok = mbar_wait_warp(&bar.q_empty[i], ((q_used >> (8 * i)) & 1) ^ 1, wc);
                    if (!ok) break;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&bar.q_full[i], q_bytes);
                        for (int bx = 0; bx < C::kBoxes; ++bx)
                            tma_load_4d(smem + C::kQOff + i * q_stride + bx * q_half, &tm_q, &bar.q_full[i], bx * 64, 0,
                                        w.row0 + t * p.tok_tile, w.h);
                    }
                    __syncwarp();
                    q_used ^= 1u << (8 * i);
                    q_at = q_at + 1 == q_slots ? 0 : q_at + 1;
                }
                it += 2 * w.cnt_max;
                const int left = w.len - (w.k0 + w.cnt_max - 1) * BN;  // keys in the part's last tile
                if (left >= BN || !ok) continue;
                const uint32_t s = (it - 1) % C::kStages;  // the part's last V
                ok = mbar_wait_warp(&bar.v_tail[s], (phases >> s) & 1, wc);
                if (!ok) continue;
                phases ^= 1u << s;
                uint8_t* tile = smem + C::kKVOff + s * C::kTileBytes;
                for (int bx = 0; bx < C::kBoxes; ++bx)
                    for (int at = left * 128 + lane * 16; at < BN * 128; at += 32 * 16)
                        *reinterpret_cast<uint4*>(tile + bx * BN * 128 + at) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
                __syncwarp();
                if (elect_one()) mbar_arrive(&bar.kv_full[s]);
                __syncwarp();
            }
            if (lane < 2) p.meta[blockIdx.x * 2 + lane] = lane == 0 ? slot0 : slot1;
            // every copy issued must land before the CTA exits: q_used holds the parity of each slot's uses
            if (lane < 4 && (lane < (int)q_slots)) {
                const uint32_t parity = (q_used >> (8 * lane)) & 1;
                drain_wait(&bar.q_full[lane], parity ^ 1, p.timeout_ns);
            }
            __syncwarp();
        } else if (!C::kOneIssuer && (warp == C::kIssuer || (NT == 2 && warp == C::kFourth))) {
            // ------------------------------------------------ MMA issuers, one per query tile
            // Each issuer walks every ring slot and releases it once, used or not. With P in columns of its own
            // S_t^{j+1} runs as soon as the softmax warps have read S_t^j, before P_t^j V; with P over S behind
            // it. (In that case the epilogue has read O_t before its threads arrive on p_full for a new unit.)
            const int t = warp == C::kIssuer ? 0 : 1;
            const uint32_t tS = tmem + t * BN, tO = tmem + C::o_col(t), tP = tmem + C::p_col(t);
            uint32_t it = 0, n_s = 0, n_p = 0;
            QRing ring(q_slots);
            bool ok = true;
            while (ok && walk.next(w)) {
                if (w.cnt_max == 0) continue;
                const int cnt = w.cnt(t);
                if (NT == 2 && t == 1 && w.cnt0 > 0) ring.next();  // tile 0's
                const uint32_t q_i = ring.at, qt = sQ + q_i * q_stride;
                if (cnt > 0) {
                    ok = mbar_wait_warp(&bar.q_full[q_i], ring.phase, wc);
                    if (!ok) break;
                    ring.next();
                    tc_fence_after();
                }
                if (NT == 2 && t == 0 && w.cnt1 > 0) ring.next();  // tile 1's
                for (int j = 0; j <= w.cnt_max && ok; ++j) {
                    const uint32_t itK = it;  // ring slot of K_j; V_j follows it
                    const uint32_t sK = itK % C::kStages, sV = (itK + C::kStages - 1) % C::kStages;
                    const uint32_t k_phase = (itK / C::kStages) & 1, v_phase = ((itK - 1) / C::kStages) & 1;
                    // with P over S the wait for P is the long one
                    const unsigned ready = !C::kSplit
                                               ? 0
                                               : look(&bar.kv_full[sK], k_phase, &bar.s_free[t], (n_s - 1) & 1, &bar.kv_full[sV],
                                                      v_phase, &bar.p_full[t], n_p & 1);
                    auto wait_s = [&]() {
                        ok = (ready & 1) || mbar_wait_warp(&bar.kv_full[sK], k_phase, wc);
                        if (C::kSplit && ok && j < cnt && n_s > 0)
                            ok = (ready & 2) || mbar_wait_warp(&bar.s_free[t], (n_s - 1) & 1, wc);
                        if (j < cnt) tc_fence_after();
                    };
                    auto wait_pv = [&]() {
                        ok = (ready & 4) || mbar_wait_warp(&bar.kv_full[sV], v_phase, wc);
                        if (ok && j <= cnt) {
                            ok = (ready & 8) || mbar_wait_warp(&bar.p_full[t], n_p & 1, wc);
                            ++n_p;
                            tc_fence_after();
                        }
                    };
                    auto issue_s = [&]() {  // S_t^j
                        if (j < cnt) {
                            if (elect_one()) {
                                const uint64_t qd = kmajor_desc(qt), kd = kmajor_desc(sKV + sK * C::kTileBytes);
#pragma unroll kIssueUnroll
                                for (int kk = 0; kk < D / 16; ++kk)
                                    mma_ss(tS, kmajor_step(qd, kk, q_half), kmajor_step(kd, kk, BN * 128), kIdescS,
                                           kk > 0 ? 1u : 0u);
                                mma_commit(&bar.s_full[t]);
                                mma_commit(&bar.kv_empty[sK]);
                                if (j == cnt - 1) mma_commit(&bar.q_empty[q_i]);  // last read of Q_t
                            }
                            ++n_s;
                        } else if (elect_one()) {
                            mma_commit(&bar.kv_empty[sK]);
                        }
                        __syncwarp();
                    };
                    auto issue_pv = [&]() {  // O_t += P_t^{j-1} V_{j-1}
                        if (j <= cnt) {
                            if (elect_one()) {
                                const uint64_t vd = vmajor_desc(sKV + sV * C::kTileBytes);
#pragma unroll kIssueUnroll
                                for (int kk = 0; kk < BN / 16; ++kk)
                                    mma_ts(tO, tP + kk * 8, vmajor_step(vd, kk), kIdescO, (j > 1 || kk > 0) ? 1u : 0u);
                                if (C::kSplit)
                                    mma_commit(&bar.pv_done[t]);
                                else if (j == cnt)
                                    mma_commit(&bar.o_full[t]);  // last product of this tile
                                mma_commit(&bar.kv_empty[sV]);
                            }
                        } else if (elect_one()) {
                            mma_commit(&bar.kv_empty[sV]);
                        }
                        __syncwarp();
                    };
                    const bool has_s = j < w.cnt_max, has_pv = j > 0;
                    if (C::kSplit) {
                        if (has_s) wait_s();
                        if (ok && has_s) issue_s();
                        if (ok && has_pv) wait_pv();
                        if (ok && has_pv) issue_pv();
                    } else {
                        // V_{j-1} is released before K_j: with an odd number of stages either producer waits on slots
                        // that the other used last, and may only see K_j's release when V_{j-1}'s is out
                        if (has_pv) wait_pv();
                        if (ok && has_pv) issue_pv();
                        if (ok && has_s) wait_s();
                        if (ok && has_s) issue_s();
                    }
                    if (j < w.cnt_max) it += 2;
                }
            }
            // every MMA this warp issued completes before TMEM is released
            if (elect_one()) {
                mma_commit(&bar.drain[t]);
                drain_wait(&bar.drain[t], 0, p.timeout_ns);
            }
            __syncwarp();
        } else if (C::kOneIssuer && warp == C::kIssuer) {
            // ------------------------------------------------ the one MMA issuer of two tiles with P over S
            // S_t^0 of every tile, then per key tile O_t += P_t^{j-1} V_{j-1} and S_t^j in turn. The epilogue has
            // read O_t before its threads arrive on p_full for a new unit.
            uint32_t it = 0, pcnt0 = 0, pcnt1 = 0;
            QRing ring(q_slots);
            bool ok = true;
            auto issue_s = [&](int t, uint32_t q_i, uint32_t sK) {
                if (elect_one()) {
                    const uint64_t qd = kmajor_desc(sQ + q_i * q_stride), kd = kmajor_desc(sKV + sK * C::kTileBytes);
#pragma unroll kIssueUnroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        mma_ss(tmem + t * BN, kmajor_step(qd, kk, q_half), kmajor_step(kd, kk, BN * 128), kIdescS,
                               kk > 0 ? 1u : 0u);
                    mma_commit(&bar.s_full[t]);
                }
                __syncwarp();
            };
            while (ok && walk.next(w)) {
                if (w.cnt_max == 0) continue;
                uint32_t sK = it % C::kStages, q_of[2];
                ok = mbar_wait_warp(&bar.kv_full[sK], (it / C::kStages) & 1, wc);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    q_of[t] = ring.at;
                    if (!ok || w.cnt(t) == 0) continue;
                    ok = mbar_wait_warp(&bar.q_full[ring.at], ring.phase, wc);
                    ring.next();
                    tc_fence_after();
                    if (ok) issue_s(t, q_of[t], sK);
                }
                if (!ok) break;
                for (int j = 1; j <= w.cnt_max && ok; ++j) {
                    const uint32_t itV = it + 1, sV = itV % C::kStages;  // V_{j-1}
                    if (elect_one()) {
                        // V before K here too; later in the key tile (behind the look at the barriers, or tile 0's
                        // products) these cost 3 %
                        if (j > 1) mma_commit(&bar.kv_empty[(it + C::kStages - 1) % C::kStages]);
                        mma_commit(&bar.kv_empty[sK]);
                        if (j == w.cnt_max) {  // every S of the part is issued
                            if (w.cnt0 > 0) mma_commit(&bar.q_empty[q_of[0]]);
                            if (NT == 2 && w.cnt1 > 0) mma_commit(&bar.q_empty[q_of[NT - 1]]);
                        }
                    }
                    __syncwarp();
                    it += 2;
                    sK = it % C::kStages;
                    const uint32_t k_phase = (it / C::kStages) & 1, v_phase = (itV / C::kStages) & 1;
                    const unsigned ready = look(&bar.kv_full[sK], k_phase, &bar.kv_full[sV], v_phase, &bar.p_full[0],
                                                pcnt0 & 1, &bar.p_full[1], pcnt1 & 1);
                    if (j < w.cnt_max) {
                        ok = (ready & 1) || mbar_wait_warp(&bar.kv_full[sK], k_phase, wc);
                        if (!ok) break;
                    }
                    ok = (ready & 2) || mbar_wait_warp(&bar.kv_full[sV], v_phase, wc);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        if (!ok || j > w.cnt(t)) continue;
                        uint32_t& pcnt = t == 0 ? pcnt0 : pcnt1;
                        ok = (ready & (t == 0 ? 4 : 8)) || mbar_wait_warp(&bar.p_full[t], pcnt & 1, wc);
                        if (!ok) continue;
                        ++pcnt;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint64_t vd = vmajor_desc(sKV + sV * C::kTileBytes);
#pragma unroll kIssueUnroll
                            for (int kk = 0; kk < BN / 16; ++kk)
                                mma_ts(tmem + C::o_col(t), tmem + t * BN + kk * 8, vmajor_step(vd, kk), kIdescO,
                                       (j > 1 || kk > 0) ? 1u : 0u);
                            if (j == w.cnt(t)) mma_commit(&bar.o_full[t]);  // last product of this tile
                        }
                        __syncwarp();
                        if (j < w.cnt(t)) issue_s(t, q_of[t], sK);
                    }
                }
                if (!ok) break;
                if (elect_one()) mma_commit(&bar.kv_empty[(it + C::kStages - 1) % C::kStages]);  // the last V
                __syncwarp();
            }
            if (elect_one()) {
                mma_commit(&bar.drain[0]);
                drain_wait(&bar.drain[0], 0, p.timeout_ns);
            }
            __syncwarp();
        }
        }
    } else {
        // ------------------------------------------------ softmax (thread = query row)
        const int t = NT == 2 ? warp >> 2 : 0;
        if constexpr (VAR == kBytes && NT == 1) {
            if (warp < 4) {
                regs_increase<C::Kernel::kOneTileRegs>();
                if (copies)
                    softmax_one<D, F16, KERNEL, true>(p, smem, bar);
                else if (warp < bar.sm_warps)
                    softmax_one<D, F16, KERNEL, false>(p, smem, bar);
            } else if (KERNEL == kMixed && warp == 4) {  // softmax warps of two-tile units
                if (copies)
                    make_factors<D, F16, KERNEL, true>(p, smem, bar);
                else
                    make_factors<D, F16, KERNEL, false>(p, smem, bar);
            } else if (KERNEL == kMixed && warp == 5) {
                if (copies)
                    issue_values<D, F16, KERNEL, true>(p, smem, bar);
                else
                    issue_values<D, F16, KERNEL, false>(p, smem, bar);
            }
        } else {
        if constexpr (C::Kernel::kRebalance) regs_increase<C::Kernel::kSoftmaxRegs>();
        if (warp < 4 * NT && (warp & 3) < bar.sm_warps) {
            const int r = (warp & 3) * 32 + lane;
            const int rows = p.tok_tile * p.G;
            const int my_tok = t * p.tok_tile + r / p.G, my_head = r % p.G;
            const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t tS = tmem + lane_off + t * BN;
            const uint32_t tO = tmem + lane_off + C::o_col(t), tP = tmem + lane_off + C::p_col(t);
            uint32_t scnt = 0, ocnt = 0;  // ocnt: phases of pv_done (split) or o_full
            bool ok = true;
            Walk<NT, KERNEL, VAR> walk(p, bar);
            Unit w;
            bool more = walk.next(w);
            // kBytes: the factor of this thread's row, and the stage of the keys' factors
            float row_c = p.c;
            int factors = 0;
            auto take_q = [&]() {
                if constexpr (VAR == kBytes) {
                    using E = Cfg8<D, F16, NT, KERNEL, false>;
                    const uint16_t* src = nullptr;
                    if (r < rows && my_tok < w.ntok) src = p.q + (w.row0 + my_tok) * p.q_sr + (w.h * p.G + my_head) * p.q_sh;
                    __syncwarp();
                    row_c = row_factor(p.c, split_row<D, F16, E::kQTmem>(src, tmem + lane_off + E::kQCol,
                                                                         smem + t * E::kPieces * E::kTileBytes, r));
                    mbar_arrive(&bar.q_full[t]);
                }
            };
            if (more && w.cnt(t) > 0) take_q();
            while (ok && more) {
                __syncwarp();  // the last use of bar.unit
                if (lane == 0) bar.unit[warp] = make_int4(w.row0, w.ntok, w.h, (w.first ? 1 : 0) + (w.last ? 2 : 0));
                const int cnt = w.cnt(t), k0 = w.k0;
                // keys this row sees, and those that the tile's first row sees
                const bool causal = VAR == kRun ? p.causal : w.causal;
                const int lim = causal ? min(w.len, w.base + my_tok + 1) : w.len;
                const int lim_first = causal ? min(w.len, w.base + t * p.tok_tile + 1) : w.len;
                // where a tree's keys begin
                const int ctx = VAR != kRun && !w.causal && p.tree != nullptr ? w.ctx : INT_MAX;
                float m_ref = -INFINITY, m_row = -INFINITY, l = 0.f;
                bool s_ready = false;
                for (int j = 0; j < cnt; ++j) {
                    const int key0 = (k0 + j) * BN;
                    ok = s_ready || mbar_wait(&bar.s_full[t], scnt & 1, wc);
                    ok = __all_sync(kFull, ok);
                    if (!ok) break;
                    ++scnt;
                    tc_fence_after();
                    uint32_t su[BN];
                    tmem_ld32_at<0>(tS + 0, su);
                    tmem_ld32_at<32>(tS + 32, su);
                    tmem_ld32_at<64>(tS + 64, su);
                    tmem_ld32_at<96>(tS + 96, su);
                    tmem_wait_ld();
                    if constexpr (VAR == kBytes) {
                        using E = Cfg8<D, F16, NT, KERNEL, false>;
                        const float4* f = reinterpret_cast<const float4*>(smem + E::kFactorOff) + factors * (BN / 4);
#pragma unroll
                        for (int i = 0; i < BN / 4; ++i) {
                            const float4 f4 = f[i];
                            const float2 a = fmul2(make_float2(__uint_as_float(su[4 * i]), __uint_as_float(su[4 * i + 1])),
                                                   make_float2(f4.x, f4.y));
                            const float2 b = fmul2(make_float2(__uint_as_float(su[4 * i + 2]), __uint_as_float(su[4 * i + 3])),
                                                   make_float2(f4.z, f4.w));
                            su[4 * i] = __float_as_uint(a.x), su[4 * i + 1] = __float_as_uint(a.y);
                            su[4 * i + 2] = __float_as_uint(b.x), su[4 * i + 3] = __float_as_uint(b.y);
                        }
                        factors = factors + 1 == E::kFactors ? 0 : factors + 1;
                    }
                    if (C::kSplit) {  // S_t is in registers: the next S_t may overwrite it
                        tc_fence_before();
                        mbar_arrive(&bar.s_free[t]);
                    }
                    if (VAR != kRun && key0 > ctx - BN) {
                        uint32_t bits[4];
                        tree_bits(p, r < rows && my_tok < w.ntok ? p.tree + (w.row0 + my_tok) * p.tree_stride : nullptr, key0, ctx,
                                  w.len, bits);
#pragma unroll
                        for (int col = 0; col < BN; ++col)
                            if (!(bits[col / 32] >> (col & 31) & 1)) su[col] = __float_as_uint(-INFINITY);
                    } else if (key0 + BN > lim_first) {
                        const int out = lim - key0;  // first column this row does not see
#pragma unroll
                        for (int col = 0; col < BN; ++col)
                            if (col >= out) su[col] = __float_as_uint(-INFINITY);
                    }
                    float mx[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        float m = fmaxf(__uint_as_float(su[16 * c]), __uint_as_float(su[16 * c + 1]));
#pragma unroll
                        for (int e = 2; e < 16; e += 2)
                            m = fmax3(m, __uint_as_float(su[16 * c + e]), __uint_as_float(su[16 * c + e + 1]));
                        mx[c] = m;
                    }
                    const float m_tile =
                        fmaxf(fmax3(fmax3(mx[0], mx[1], mx[2]), mx[3], mx[4]), fmax3(mx[5], mx[6], mx[7])) * row_c;
                    m_row = fmaxf(m_row, m_tile);
                    float m_new = m_ref;
                    if (m_tile > m_ref + kRescaleThreshold) m_new = m_tile;
                    const bool moved = m_new != m_ref;
                    const float alpha = moved ? ex2(m_ref - m_new) : 1.f;  // 0 when m_ref = -inf
                    const bool rescale = j > 0 && __any_sync(kFull, moved && m_ref != -INFINITY);
                    auto rescale_o = [&]() {
#pragma unroll 1  // rare, and unrolled it costs the key loop its registers
                        for (int c0 = 0; c0 < D; c0 += 32) {
                            uint32_t ov[32];
                            tmem_ld32(tO + c0, ov);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; i += 2) {
                                const float2 r2 = fmul2(make_float2(__uint_as_float(ov[i]), __uint_as_float(ov[i + 1])),
                                                        make_float2(alpha, alpha));
                                ov[i] = __float_as_uint(r2.x);
                                ov[i + 1] = __float_as_uint(r2.y);
                            }
                            tmem_st32(tO + c0, ov);
                        }
                    };
                    // without split P the previous P V precedes this S in the MMA stream
                    if (!C::kSplit && rescale) rescale_o();
                    m_ref = m_new;
                    const float neg_m = (m_ref == -INFINITY) ? 0.f : -m_ref;
                    const float2 cc2 = make_float2(row_c, row_c), nm2 = make_float2(neg_m, neg_m);
                    float2 suma = make_float2(0.f, 0.f), sumb = make_float2(0.f, 0.f);
                    if (C::kSplit) {
                        // Looking at a barrier takes some 130 cycles. The product of tile j-1 has mostly ended by
                        // now, and S_{j+1} before this tile does: both are looked at early, beside other work.
                        bool o_ready = false;
#pragma unroll
                        for (int i = 0; i < BN / 2; ++i) {
                            if (i == BN / 2 - 16 && j > 0) o_ready = mbar_test(&bar.pv_done[t], ocnt & 1);
                            const float2 x = ffma2(make_float2(__uint_as_float(su[2 * i]), __uint_as_float(su[2 * i + 1])),
                                                   cc2, nm2);
                            const float2 pp = make_float2(ex2(x.x), ex2(x.y));
                            if (i & 1)
                                sumb = fadd2(sumb, pp);
                            else
                                suma = fadd2(suma, pp);
                            su[i] = pack_h16<F16>(pp.x, pp.y);
                        }
                        if (j > 0) {  // the product of tile j-1 has read P_t and written O_t
                            ok = o_ready || mbar_wait(&bar.pv_done[t], ocnt & 1, wc);
                            ok = __all_sync(kFull, ok);
                            if (!ok) break;
                            ++ocnt;
                            tc_fence_after();
                            if (rescale) rescale_o();
                        }
                        tmem_st32_at<0>(tP + 0, su);
                        tmem_st32_at<32>(tP + 32, su);
                        s_ready = j + 1 < cnt && mbar_test(&bar.s_full[t], scnt & 1);
                    } else {
#pragma unroll
                        for (int c0 = 0; c0 < BN; c0 += 32) {
                            uint32_t pk[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float2 x = ffma2(
                                    make_float2(__uint_as_float(su[c0 + 2 * i]), __uint_as_float(su[c0 + 2 * i + 1])), cc2,
                                    nm2);
                                const float2 pp = make_float2(ex2(x.x), ex2(x.y));
                                if (i & 1)
                                    sumb = fadd2(sumb, pp);
                                else
                                    suma = fadd2(suma, pp);
                                pk[i] = pack_h16<F16>(pp.x, pp.y);
                            }
                            tmem_st16(tS + c0 / 2, pk);
                        }
                    }
                    l = l * alpha + ((suma.x + suma.y) + (sumb.x + sumb.y));
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(&bar.p_full[t]);
                }
                if (!ok) break;
                if constexpr (VAR == kBytes)
                    factors = (factors + w.cnt_max - cnt) % Cfg8<D, F16, NT, KERNEL, false>::kFactors;  // of tiles that only the other saw
                more = walk.next(w);  // while the last product runs
                if (more && w.cnt(t) > 0) take_q();  // every product with this unit's has been waited for
                if (cnt > 0) {
                    ok = mbar_wait(C::kSplit ? &bar.pv_done[t] : &bar.o_full[t], ocnt & 1, wc);
                    ok = __all_sync(kFull, ok);
                    if (!ok) break;
                    ++ocnt;
                    tc_fence_after();
                }
                __syncwarp();
                const int4 u = bar.unit[warp];
                finish_row<D, F16, C::Kernel::kTiles>(p, u, t, r, my_tok, my_head, rows, cnt, tO, m_ref, m_row, l);
                tc_fence_before();
            }
        }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // Every copy issued must land before the CTA exits. The issuers have waited for each, unless a wait ran out.
    if (threadIdx.x == 0 && bar.abort_flag != 0) {
        if constexpr (VAR == kBytes) {
            using E = Cfg8<D, F16, NT, KERNEL, false>;
            using S = Cfg8<D, F16, NT, KERNEL, NT == 1>;
            drain_codes(bar, copies ? S::kKeys : E::kKeys, copies ? S::kValues : E::kValues, p.timeout_ns);
        } else {
            drain_ring(bar, C::kStages, p.timeout_ns);
        }
    }
}

template <int D, bool F16, int KERNEL, int VAR>
__global__ void __launch_bounds__(Shape<D, KERNEL, VAR>::kThreads, Shape<D, KERNEL, VAR>::kPerSm)
    paged_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const PagedDev p) {
    using Kernel = Shape<D, KERNEL, VAR>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Shared& bar = *reinterpret_cast<Shared*>(smem + Kernel::kTilesBytes);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) bar.abort_flag = 0;
    if (warp == 0) {
        tmem_alloc(&bar.tmem_base, Kernel::kTmemCols);
        tmem_relinquish();
        if (elect_one()) {
            prefetch_tmap(&tm_q);
            prefetch_tmap(&tm_k);
            prefetch_tmap(&tm_v);
        }
        __syncwarp();
    }
    tc_fence_before();
    // The next kernel may come once every CTA has its tensor memory, or it could take it and wait for this one.
    __syncthreads();
    grid_dep_launch();
    // No global memory is touched above: from here on the previous kernel must be complete.
    grid_dep_wait();
    locate<Kernel::kTiles, Kernel::kThreads, VAR>(p, bar);
    __syncthreads();
    if constexpr (KERNEL == kMixed) {
        if (bar.pair)
            work<D, F16, 2, KERNEL, VAR>(tm_q, tm_k, tm_v, p, smem, bar);
        else
            work<D, F16, 1, KERNEL, VAR>(tm_q, tm_k, tm_v, p, smem, bar);
    } else {
        work<D, F16, 1, KERNEL, VAR>(tm_q, tm_k, tm_v, p, smem, bar);
    }
    if (warp == 0) tmem_dealloc(bar.tmem_base, Kernel::kTmemCols);
}

// ---------------------------------------------------------------- merging parts
struct CombineArgs {
    float* part;
    const int4* meta;
    int ctas;
    int tiles, rows;     // tiles of a slot, rows of a tile
    int tok_tile, G, T;
    uint8_t* o;
    float* lse;
    long long o_sr, o_sh;
};

constexpr int kCombineThreads = 256;

// Merges the units that were cut. The CTA that wrote a unit's last part names the unit: its first part is in
// slot 1 of the nearest CTA before that one that has one, the parts between in the slots 0. A thread takes 16
// columns of a row, threads side by side the rows; the parts are merged as tiles are, in the order of the
// keys.
// How many units there are and how large is known here only. With SHARE every block counts the work (in
// blocks' worth of threads, by the units in order) and takes its shares of it; without, block (e, y) takes the
// y-th share of the unit that CTA e ended, if there is one. SHARE is for units that may have more than 4
// shares (two tiles at d = 128 have 8), where most blocks would find nothing to do: a step of 16 decoding
// sequences and a 512-row chunk takes 70.1 us without SHARE and 67.8 with it, 16 chunks of 40 rows 44.2 and
// 41.4. With up to 4, blocks that know their unit start sooner: one token takes 10.5 us and 11.3 with SHARE,
// at d = 64 16 chunks of 40 rows 28.6 and 30.2, 8 chunks of 448 rows 39.6 and 40.0.
template <int D, bool F16, bool SHARE>
__global__ void __launch_bounds__(kCombineThreads) paged_combine_kernel(const CombineArgs a) {
    constexpr int kGroups = D / 16, kWarps = kCombineThreads / 32;
    grid_dep_launch();
    grid_dep_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ctas = SHARE ? a.ctas : blockIdx.x + 1;  // that the block looks at
    const int words = (ctas + 31) / 32;
    extern __shared__ int4 s_units[];  // slot 0 of every CTA
    // bit c of has0 / has1: CTA c's slot 0 / 1 holds a part
    unsigned* has0 = reinterpret_cast<unsigned*>(s_units + 32 * words);
    unsigned* has1 = has0 + words;
    int* sums = reinterpret_cast<int*>(has1 + words);  // shares of 32 CTAs' units
    int* ends = sums + words;                          // of the CTAs of a word up to this one
    int4 own = make_int4(kNone, 0, 0, 0);
    if (!SHARE) own = a.meta[(ctas - 1) * 2];  // read along with the others
    for (int w = warp; w < words; w += kWarps) {
        const int c = w * 32 + lane, at = min(c, ctas - 1) * 2;
        const int4 m = a.meta[at];
        const int other = a.meta[at + 1].x;
        const unsigned b0 = __ballot_sync(kFull, c < ctas && m.x != kNone);
        const unsigned b1 = __ballot_sync(kFull, c < ctas && other != kNone);
        if (lane == 0) {
            has0[w] = b0;
            has1[w] = b1;
        }
        if (SHARE) {
            int x = c < ctas && m.x == kLast ? (m.z * a.G * kGroups + kCombineThreads - 1) / kCombineThreads : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(kFull, x, o);
                if (lane >= o) x += u;
            }
            s_units[c] = m;
            ends[c] = x;
            if (lane == 31) sums[w] = x;
        }
    }
    if (!SHARE && own.x != kLast) return;
    __syncthreads();
    int total = SHARE ? 0 : 1;
    if (SHARE)
        for (int w = 0; w < words; ++w) total += sums[w];
    for (int share = SHARE ? blockIdx.x : 0; share < total; share += gridDim.x) {
        int e = ctas - 1, left = blockIdx.y;  // the unit that CTA e ended, which of its shares
        int4 unit = own;
        if (SHARE) {
            int w = 0;
            left = share;
            while (left >= sums[w]) left -= sums[w++];
            const int c = __ffs(__ballot_sync(kFull, ends[w * 32 + lane] > left)) - 1;
            e = w * 32 + c;
            if (c > 0) left -= ends[e - 1];
            unit = s_units[e];
        }
        int word = e / 32;
        unsigned before = has1[word] & ((1u << (e & 31)) - 1);
        while (before == 0 && word > 0) before = has1[--word];
        if (before == 0) continue;
        const int bit = 31 - __clz(before);
        int slot = (word * 32 + bit) * 2 + 1;  // of the part to come
        unsigned behind = has0[word] & ~(0xffffffffu >> (31 - bit));  // the word's slots 0 after it
        const int rows = unit.z * a.G, i = left * kCombineThreads + tid;
        if (i >= rows * kGroups) continue;
        const int group = i / rows, row_of = i % rows;
        const int t = row_of / a.rows, r = row_of % a.rows;
        const int tok = t * a.tok_tile + r / a.G;
        float M = -INFINITY, L = 0.f, Lo = 0.f, out[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) out[c] = 0.f;
        // One pass with a running maximum, four parts' loads in flight at a time. Entries behind the last part
        // repeat it; their weight is 0.
        bool more = true;
        while (more) {
            float4 head[4], o[4][4];
            int from[4], parts = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                from[q] = slot;
                if (!more) continue;
                parts = q + 1;
                more = slot != e * 2;
                if (!more) continue;
                while (behind == 0) behind = has0[++word];
                slot = (word * 32 + __ffs(behind) - 1) * 2;
                behind &= behind - 1;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4* rec = record(a.part, from[q], a.tiles, t, a.rows, D) + r;
                head[q] = rec[0];
#pragma unroll
                for (int c = 0; c < 4; ++c) o[q][c] = rec[(1 + group * 4 + c) * a.rows];
            }
#pragma unroll
            for (int q = 1; q < 4; ++q)
                if (q >= parts) head[q].x = -INFINITY;
            const float m = fmaxf(fmaxf(M, fmaxf(head[0].x, head[1].x)), fmaxf(head[2].x, head[3].x));
            const float was = M == -INFINITY ? 0.f : ex2(M - m);
            M = m;
            L *= was;
            Lo *= was;
#pragma unroll
            for (int c = 0; c < 16; ++c) out[c] *= was;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (head[q].x == -INFINITY) continue;  // no key of this row in the part: its o was not written
                const float f = ex2(head[q].x - m);
                L = fmaf(f, head[q].y, L);
                Lo = fmaf(f, head[q].z, Lo);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    out[4 * c] = fmaf(f, o[q][c].x, out[4 * c]);
                    out[4 * c + 1] = fmaf(f, o[q][c].y, out[4 * c + 1]);
                    out[4 * c + 2] = fmaf(f, o[q][c].z, out[4 * c + 2]);
                    out[4 * c + 3] = fmaf(f, o[q][c].w, out[4 * c + 3]);
                }
            }
        }
        const float inv = Lo > 0.f ? 1.f / Lo : 0.f;
        const long long row = unit.y + tok, head = unit.w * a.G + r % a.G;
        uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.o) + row * a.o_sr + head * a.o_sh + group * 16);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            uint4 v;
            v.x = pack_h16<F16>(out[8 * q + 0] * inv, out[8 * q + 1] * inv);
            v.y = pack_h16<F16>(out[8 * q + 2] * inv, out[8 * q + 3] * inv);
            v.z = pack_h16<F16>(out[8 * q + 4] * inv, out[8 * q + 5] * inv);
            v.w = pack_h16<F16>(out[8 * q + 6] * inv, out[8 * q + 7] * inv);
            dst[q] = v;
        }
        if (group == 0) a.lse[head * a.T + row] = row_lse(M, L);
    }
}

// ---------------------------------------------------------------- host side
// The tile shape of a call. One tile per unit while the rows that a sequence is expected to bring fit
// it, so that decode does not carry an empty second tile; two beyond.
struct Plan {
    int kernel, tiles, tok_tile, rows, ctas, num_sms;
    size_t meta_bytes, bytes;
};

Plan plan_of(const attn_paged_params& p, int num_sms, int var) {
    const int G = p.num_q_heads / p.num_kv_heads;
    Plan pl;
    pl.tiles = (long long)p.max_q * G > BM ? 2 : 1;
    pl.num_sms = num_sms;
    pl.tok_tile = BM / G;
    if (pl.tiles == 1 && p.max_q < pl.tok_tile) pl.tok_tile = p.max_q;
    pl.rows = pl.tok_tile * G;
    const bool few = var == kRun && p.d == 128 && pl.rows <= kFewRows && (long long)p.max_pages * p.page_size <= kFewKeys;
    pl.kernel = pl.tiles == 2 ? kMixed : few ? kFew : kOne;
    pl.ctas = num_sms * (var != kBytes && (pl.kernel == kFew || (pl.kernel == kOne && p.d == 64)) ? 2 : 1);  // Shape::kPerSm
    // the workspace has room for either one-tile kernel, so that its size does not go by the table's, and is
    // the same for every variant
    const int room = num_sms * (pl.tiles == 1 && (p.d == 64 || pl.rows <= kFewRows) ? 2 : 1);
    pl.meta_bytes = ((size_t)room * 2 * sizeof(int4) + 255) / 256 * 256;
    pl.bytes = pl.meta_bytes + (size_t)room * 2 * pl.tiles * pl.rows * (p.d + 4) * sizeof(float);
    return pl;
}

// kBytes: a score is (sum of products of pieces of Q and codes) * (key's scale 2^k) * (row's 2^e) * c in this order, and the sum
// may reach 2^28 where k reaches 119. So 2^-bias of the latter two goes onto the keys' scales, as much as leaves c * 2^bias * 2^e
// finite for every e, and no more than is needed. The product with a key's factor then stays within fp32 for k up to 100 +
// bias: up to 113 for a scale of 1 / 8 and less, 110 for 1.
int key_bias_of(float c) { return (int)std::min(19.f, std::max(0.f, std::floor(127.f - kMostRowExponent - std::log2(c)))); }

// 4-D map of 16-bit elements over the given extents, dimension 0 contiguous, 64-column boxes.
// Rows of 64 columns that do not follow one another (pages that hold [slot, head, d]) are fetched in
// 128-byte pieces, or half of every fetch would be another head's row: 64 sequences of 4096 keys at d = 64 took
// 112 us with 256-byte promotion and take 86 (80 % of the measured HBM). At d = 128, 256 bytes are a row, and
// 128-byte promotion is 6 % slower with 16-token pages.
CUresult encode(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* m, int32_t dtype, const void* base,
                const cuuint64_t (&dims)[4], const int64_t (&st)[3], cuuint32_t box1, cuuint32_t box2) {
    cuuint64_t strides[3];
    for (int i = 0; i < 3; ++i) strides[i] = dims[i + 1] > 1 ? (cuuint64_t)st[i] * 2 : 16;  // unread over an extent of 1
    const cuuint32_t box[4] = {64, box1, box2, 1}, es[4] = {1, 1, 1, 1};
    return enc(m, dtype == ATTN_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
               const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               dims[0] == 64 && st[0] != 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// The same for caches of codes: whole rows of bytes, swizzled as the products (keys) or the converters read them, strides
// in bytes.
CUresult encode_codes(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* m, const void* base, const cuuint64_t (&dims)[4],
                      const int64_t (&st)[3], cuuint32_t box_rows, bool keys) {
    cuuint64_t strides[3];
    for (int i = 0; i < 3; ++i) strides[i] = dims[i + 1] > 1 ? (cuuint64_t)st[i] : 16;
    const cuuint32_t box[4] = {(cuuint32_t)dims[0], box_rows, 1, 1}, es[4] = {1, 1, 1, 1};
    const CUtensorMapSwizzle swizzle = dims[0] == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                       : keys         ? CU_TENSOR_MAP_SWIZZLE_64B
                                                      : CU_TENSOR_MAP_SWIZZLE_NONE;
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

template <int D, bool F16, int KERNEL, int VAR>
cudaError_t launch_tc(const CUtensorMap (&maps)[3], const PagedDev& p, int grid, cudaStream_t s) {
    using Kernel = Shape<D, KERNEL, VAR>;
    const cudaError_t e = cudaFuncSetAttribute(paged_tc_kernel<D, F16, KERNEL, VAR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Kernel::kSmemBytes);
    if (e != cudaSuccess) return e;
    // kMixed of kBytes starts when every SM is free, so that its CTAs mostly come to lie in their order (locate): started early,
    // one by one as SMs fall free, both kinds end up side by side (24 trees over an 8-bit cache 304 us, 174 in order).
    return launch_chained(!(VAR == kBytes && KERNEL == kMixed), paged_tc_kernel<D, F16, KERNEL, VAR>, dim3(grid),
                          dim3(Kernel::kThreads), Kernel::kSmemBytes, s, maps[0], maps[1], maps[2], p);
}

template <int D, bool F16, int VAR>
cudaError_t launch_both(const CUtensorMap (&maps)[3], const PagedDev& p, const Plan& pl, int grid, cudaStream_t s) {
    // Held from a call's first launch to its last, so that calls of several host threads on one stream may share
    // a workspace: the parts that one call leaves there are merged before the next call's are written.
    std::lock_guard<std::mutex> lock(paged_launch_mutex());
    cudaError_t e;
    if (pl.kernel == kMixed) {
        e = launch_tc<D, F16, kMixed, VAR>(maps, p, grid, s);
    } else if (pl.kernel == kFew) {
        if constexpr (D == 128 && VAR == kRun)
            e = launch_tc<128, F16, kFew, VAR>(maps, p, grid, s);
        else
            e = cudaErrorInvalidValue;  // not planned
    } else {
        e = launch_tc<D, F16, kOne, VAR>(maps, p, grid, s);
    }
    if (e != cudaSuccess) return e;
    CombineArgs a{};
    a.part = p.part;
    a.meta = p.meta;
    a.ctas = grid;
    a.tiles = pl.tiles;
    a.rows = pl.rows;
    a.tok_tile = p.tok_tile;
    a.G = p.G;
    a.T = p.T;
    a.o = p.o;
    a.lse = p.lse;
    a.o_sr = p.o_sr;
    a.o_sh = p.o_sh;
    const int words = (grid + 31) / 32, most = (pl.tiles * pl.rows * (D / 16) + kCombineThreads - 1) / kCombineThreads;
    const size_t smem = 32 * words * sizeof(int4) + 35 * words * sizeof(int);
    if constexpr (D == 128)
        if (most > 4)
            return launch_pdl(paged_combine_kernel<D, F16, true>, dim3(min(grid * most, 2 * pl.num_sms)), dim3(kCombineThreads),
                              smem, s, a);
    return launch_pdl(paged_combine_kernel<D, F16, false>, dim3(grid, most), dim3(kCombineThreads), smem, s, a);
}

// What a variant brings besides the call itself.
struct Extra {
    const int32_t* mask = nullptr;  // bits of a tree's rows
    int64_t mask_stride = 0;
    int32_t words = 0;
    const void *k_scale = nullptr, *v_scale = nullptr;
    int64_t k_scale_stride[2] = {}, v_scale_stride[2] = {};
};

template <int VAR>
attn_status_t launch_variant(const attn_paged_params& p, const Extra& x, const LaunchCommon& lc, cudaStream_t s) {
    PFN_cuTensorMapEncodeTiled_v12000 enc;
    const attn_status_t st = map_encoder(&enc);
    if (st != ATTN_OK) return st;
    const Plan pl = plan_of(p, lc.num_sms, VAR);
    const int G = p.num_q_heads / p.num_kv_heads;
    CUtensorMap maps[3];
    // q as (column, head in the group, row, key/value head); the caches as (column, slot, head, page)
    const cuuint64_t qd[4] = {(cuuint64_t)p.d, (cuuint64_t)G, (cuuint64_t)p.total_q, (cuuint64_t)p.num_kv_heads};
    const int64_t qs[3] = {p.q_stride[1], p.q_stride[0], p.q_stride[1] * G};
    const cuuint64_t cd[4] = {(cuuint64_t)p.d, (cuuint64_t)p.page_size, (cuuint64_t)p.num_kv_heads, (cuuint64_t)p.num_pages};
    const int64_t ks[3] = {p.k_stride[2], p.k_stride[1], p.k_stride[0]}, vs[3] = {p.v_stride[2], p.v_stride[1], p.v_stride[0]};
    const cuuint32_t box_rows = (cuuint32_t)(p.page_size < BN ? p.page_size : BN);
    CUresult r = encode(enc, &maps[0], p.dtype, p.q, qd, qs, (cuuint32_t)G, (cuuint32_t)pl.tok_tile);
    if (VAR == kBytes) {
        if (r == CUDA_SUCCESS) r = encode_codes(enc, &maps[1], p.k_cache, cd, ks, box_rows, true);
        if (r == CUDA_SUCCESS) r = encode_codes(enc, &maps[2], p.v_cache, cd, vs, box_rows, false);
    } else {
        if (r == CUDA_SUCCESS) r = encode(enc, &maps[1], p.dtype, p.k_cache, cd, ks, box_rows, 1);
        if (r == CUDA_SUCCESS) r = encode(enc, &maps[2], p.dtype, p.v_cache, cd, vs, box_rows, 1);
    }
    if (r != CUDA_SUCCESS) return report_error(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled(attn_paged) failed with %d", (int)r);
    PagedDev a{};
    a.B = p.num_seqs;
    a.G = G;
    a.Hkv = p.num_kv_heads;
    a.T = p.total_q;
    a.tok_tile = pl.tok_tile;
    a.num_pages = p.num_pages;
    a.page_size = p.page_size;
    while ((1 << a.shift) < p.page_size) ++a.shift;
    a.max_pages = p.max_pages;
    a.causal = p.causal;
    const int bias = VAR == kBytes ? key_bias_of(p.scale * kLog2e) : 0;
    a.c = std::ldexp(p.scale * kLog2e, bias);
    a.key_bias = std::ldexp(1.f, -bias);
    a.cu_q = p.cu_q;
    a.kv_len = p.kv_len;
    a.table = p.block_table;
    a.table_stride = p.table_stride;
    a.o = static_cast<uint8_t*>(p.o);
    a.lse = p.lse;
    a.o_sr = p.o_stride[0];
    a.o_sh = p.o_stride[1];
    a.o_wide = ((reinterpret_cast<uintptr_t>(p.o) | (uintptr_t)(p.total_q > 1 ? p.o_stride[0] * 2 : 0) |
                 (uintptr_t)(p.num_q_heads > 1 ? p.o_stride[1] * 2 : 0)) & 31) == 0;
    a.meta = static_cast<int4*>(p.workspace);
    a.part = reinterpret_cast<float*>(static_cast<char*>(p.workspace) + pl.meta_bytes);
    a.err = lc.err;
    a.timeout_ns = lc.timeout_ns;
    a.stall_after = lc.stall_after;
    a.tree = reinterpret_cast<const uint32_t*>(x.mask);
    a.tree_stride = x.mask_stride;
    a.tree_words = x.words;
    a.tree_nodes = x.mask ? 32 * x.words : p.causal ? 0 : INT_MAX;
    a.k_scale = static_cast<const uint8_t*>(x.k_scale);
    a.v_scale = static_cast<const uint8_t*>(x.v_scale);
    a.q = static_cast<const uint16_t*>(p.q);
    a.q_sr = p.q_stride[0];
    a.q_sh = p.q_stride[1];
    a.ks_page = x.k_scale_stride[0];
    a.ks_head = x.k_scale_stride[1];
    a.vs_page = x.v_scale_stride[0];
    a.vs_head = x.v_scale_stride[1];
    const bool f16 = p.dtype == ATTN_F16;
    const cudaError_t e = p.d == 64 ? (f16 ? launch_both<64, true, VAR>(maps, a, pl, pl.ctas, s)
                                           : launch_both<64, false, VAR>(maps, a, pl, pl.ctas, s))
                                    : (f16 ? launch_both<128, true, VAR>(maps, a, pl, pl.ctas, s)
                                           : launch_both<128, false, VAR>(maps, a, pl, pl.ctas, s));
    return e == cudaSuccess ? ATTN_OK : report_error(ATTN_ERR_CUDA, "attn_paged launch: %s", cudaGetErrorString(e));
}

}  // namespace
}  // namespace attn
