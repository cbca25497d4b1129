// attn_paged.cu — attention of a ragged batch of new tokens over a paged cache, on
// the tensor cores.
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
#include <cuda_bf16.h>

#include <cfloat>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "internal.h"
#include "ptx.cuh"

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

template <int D, int KERNEL>
struct Shape {
    static constexpr int kTiles = KERNEL == kMixed ? 2 : 1;  // of a unit, at most
    static constexpr int kPerSm = KERNEL == kFew || (KERNEL == kOne && D == 64) ? 2 : 1;
    static constexpr int kFirst = 4 * kTiles;  // the first warp behind the softmax warps
    static constexpr int kThreads = KERNEL == kMixed ? 384 : 256;
    // shared memory for Q, K and V tiles
    static constexpr int kTilesBytes = (KERNEL == kFew ? 104 : kPerSm == 2 ? 96 : 224) * 1024;
    static constexpr int kSmemBytes = kTilesBytes + 2048 + 1024;  // barriers and schedule + alignment slack
    static_assert(kPerSm * (kSmemBytes + 1024) <= 228 * 1024, "shared memory");
    static constexpr uint32_t kTmemCols = 512 / kPerSm;
    // registers per thread after the rebalance: the softmax warps hold a row of scores each
    static constexpr bool kRebalance = KERNEL == kMixed || kPerSm == 2;
    static constexpr int kSoftmaxRegs = KERNEL != kMixed ? 184 : D == 64 ? 192 : 200;
    static constexpr int kOtherRegs = KERNEL != kMixed ? 72 : D == 64 ? 120 : 104;
    static_assert(KERNEL != kMixed ? kSoftmaxRegs + kOtherRegs <= 2 * 128 : 2 * kSoftmaxRegs + kOtherRegs <= 3 * 168,
                  "register split");
};

// A CTA of the kernel KERNEL that works on units of NT tiles.
template <int D, int NT, int KERNEL>
struct Cfg {
    using Kernel = Shape<D, KERNEL>;
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

struct PagedDev {
    int B, G, Hkv, T;
    int tok_tile;     // tokens of a tile: its rows are tok_tile * G
    int num_pages, page_size, shift, max_pages;
    int causal;
    float c;          // scale * log2(e)
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
    uint64_t s_full[2], p_full[2], o_full[2], s_free[2], pv_done[2];
    uint64_t drain[2];
    long long x0, x1;      // this CTA's piece of the line
    Place first;           // the unit that holds x0; u0 = -1 if there is none
    Place place[12];       // of each warp
    int4 unit[12];         // of each softmax warp, the unit it is in: first row of q, tokens, key/value
                           // head, 1 if it holds the first key tile + 2 if the last
    long long scan[2][12]; // per warp: its sequences' cost on either line
    int pair;              // whether this CTA works on two-tile units
    int widest[12], sm_warps;  // most rows of a one-tile unit; softmax warps of a tile that hold rows
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

// Keys that the last of a sequence's first `tok` rows sees.
__device__ __forceinline__ int visible(const PagedDev& p, const Seq& s, int tok) {
    return p.causal ? max(0, s.len - s.n + tok) : s.len;
}

// Cost of the first i units of one head (all but the sequence's last unit are full, so their visible
// keys grow by `step` rows each, from where they are positive on).
__device__ __forceinline__ long long cost_before(const PagedDev& p, const Seq& s, int step, long long i) {
    if (!p.causal) return i * (s.len + kUnitCost);
    const long long base = s.len - s.n;
    const long long m = base >= 0 ? 1 : -base / step + 1;  // the first unit (from 1) with a visible key
    long long sum = i * kUnitCost;
    if (i >= m) sum += (i - m + 1) * base + step * (i * (i + 1) / 2 - m * (m - 1) / 2);
    return sum;
}

__device__ __forceinline__ long long head_cost(const PagedDev& p, const Seq& s, int step) {
    if (s.n == 0) return 0;
    const int units = (s.n + step - 1) / step;
    return cost_before(p, s, step, units - 1) + visible(p, s, s.n) + kUnitCost;
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
template <int NT, int THREADS>
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
        per_head = head_cost(p, s, two ? 2 * p.tok_tile : p.tok_tile);
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
        const float c0 = (float)done[0], c1 = (float)done[1] * kPairCost;
        int n0 = done[0] == 0 ? 0 : max(1, (int)(n * (c0 / (c0 + c1)) + 0.5f));
        if (done[1] > 0) n0 = min(n0, n - 1);
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
                if (cost_before(p, s, step, mid) <= in_head)
                    lo = mid;
                else
                    hi = mid;
            }
            sh.first = Place{begin + h * per_head + cost_before(p, s, step, lo), b0 + tid, h, lo, s};
        }
        if ((pair ? done[1] : done[0]) > x0) break;
    }
    if (tid == 0) {
        sh.x0 = x0;
        sh.x1 = x1;
        sh.pair = pair;
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
    __device__ __forceinline__ int cnt(int t) const { return t == 0 ? cnt0 : cnt1; }
};

// Walks this CTA's units of NT tiles in order. Every warp role walks for itself and finds the same units;
// its place is kept in shared memory, since the softmax warps need their registers for a row of scores.
// In the mixed kernel sequences of the other kind are passed over.
template <int NT, int KERNEL>
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
            const int keys = visible(p, s, tok0 + w.ntok);
            const int tiles = (keys + BN - 1) / BN;
            const long long end = at.u0 + keys + kUnitCost;
            const int k0 = x0 <= at.u0 ? 0 : min(tiles, (int)((x0 - at.u0 + BN / 2) / BN));
            const int k1 = x1 >= end ? tiles : min(tiles, (int)((x1 - at.u0 + BN / 2) / BN));
            mine = k0 < k1 || (tiles == 0 && at.u0 >= x0);
            w.b = at.b;
            w.h = at.h;
            w.row0 = s.row0 + tok0;
            w.len = s.len;
            w.base = p.causal ? s.len - s.n + tok0 : s.len - 1;
            w.k0 = k0;
            w.first = k0 == 0;
            w.last = k1 == tiles;
            w.cnt_max = k1 - k0;
            w.cnt0 = w.cnt_max;
            w.cnt1 = 0;
            if (NT == 2 && w.ntok > p.tok_tile) {  // causal: tile 0's rows may see fewer tiles
                w.cnt1 = w.cnt_max;
                w.cnt0 = max(0, min(k1, (visible(p, s, tok0 + p.tok_tile) + BN - 1) / BN) - k0);
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

// The work of a CTA on units of NT tiles, from the located piece of the line to its end.
template <int D, bool F16, int NT, int KERNEL>
__device__ __forceinline__ void work(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                     const PagedDev& p, uint8_t* smem, Shared& bar) {
    using C = Cfg<D, NT, KERNEL>;
    constexpr uint32_t kIdescS = idesc_h16(BM, BN, false, false, F16);
    constexpr uint32_t kIdescO = idesc_h16(BM, D, false, true, F16);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const WaitCtl wc{p.err, &bar.abort_flag, p.timeout_ns};
    if (threadIdx.x == 0) {
        const uint32_t rows = 32u * (uint32_t)bar.sm_warps;  // softmax threads of a tile
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bar.q_full[i], 1);
            mbar_init(&bar.q_empty[i], 1);
        }
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&bar.kv_full[s], 1);
            mbar_init(&bar.kv_empty[s], C::kIssuers);
            mbar_init(&bar.v_tail[s], 1);
        }
        for (int t = 0; t < NT; ++t) {
            mbar_init(&bar.s_full[t], 1);
            mbar_init(&bar.p_full[t], rows);
            mbar_init(&bar.o_full[t], 1);
            mbar_init(&bar.s_free[t], rows);
            mbar_init(&bar.pv_done[t], 1);
            mbar_init(&bar.drain[t], 1);
        }
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
        Walk<NT, KERNEL> walk(p, bar);
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
    } else {
        if constexpr (C::Kernel::kRebalance) regs_increase<C::Kernel::kSoftmaxRegs>();
        // ------------------------------------------------ softmax (thread = query row)
        const int t = NT == 2 ? warp >> 2 : 0;
        if (warp < 4 * NT && (warp & 3) < bar.sm_warps) {
            const int r = (warp & 3) * 32 + lane;
            const int rows = p.tok_tile * p.G;
            const int my_tok = t * p.tok_tile + r / p.G, my_head = r % p.G;
            const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t tS = tmem + lane_off + t * BN;
            const uint32_t tO = tmem + lane_off + C::o_col(t), tP = tmem + lane_off + C::p_col(t);
            uint32_t scnt = 0, ocnt = 0;  // ocnt: phases of pv_done (split) or o_full
            bool ok = true;
            Walk<NT, KERNEL> walk(p, bar);
            Unit w;
            bool more = walk.next(w);
            while (ok && more) {
                __syncwarp();  // the last use of bar.unit
                if (lane == 0) bar.unit[warp] = make_int4(w.row0, w.ntok, w.h, (w.first ? 1 : 0) + (w.last ? 2 : 0));
                const int cnt = w.cnt(t), k0 = w.k0;
                // keys this row sees, and those that the tile's first row sees
                const int lim = p.causal ? min(w.len, w.base + my_tok + 1) : w.len;
                const int lim_first = p.causal ? min(w.len, w.base + t * p.tok_tile + 1) : w.len;
                float m_ref = -INFINITY, m_row = -INFINITY, l = 0.f;
                bool s_ready = false;
                for (int j = 0; j < cnt; ++j) {
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
                    if (C::kSplit) {  // S_t is in registers: the next S_t may overwrite it
                        tc_fence_before();
                        mbar_arrive(&bar.s_free[t]);
                    }
                    const int key0 = (k0 + j) * BN;
                    if (key0 + BN > lim_first) {
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
                        fmaxf(fmax3(fmax3(mx[0], mx[1], mx[2]), mx[3], mx[4]), fmax3(mx[5], mx[6], mx[7])) * p.c;
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
                    const float2 cc2 = make_float2(p.c, p.c), nm2 = make_float2(neg_m, neg_m);
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
                more = walk.next(w);  // while the last product runs
                if (cnt > 0) {
                    ok = mbar_wait(C::kSplit ? &bar.pv_done[t] : &bar.o_full[t], ocnt & 1, wc);
                    ok = __all_sync(kFull, ok);
                    if (!ok) break;
                    ++ocnt;
                    tc_fence_after();
                }
                __syncwarp();
                const int4 u = bar.unit[warp];
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
                    float4* rec = record(p.part, blockIdx.x * 2 + (first ? 1 : 0), C::Kernel::kTiles, t, rows, D);
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
                tc_fence_before();
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // Every copy issued must land before the CTA exits. The issuers have waited for each, unless a wait ran out.
    if (threadIdx.x == 0 && bar.abort_flag != 0) drain_ring(bar, C::kStages, p.timeout_ns);
}

template <int D, bool F16, int KERNEL>
__global__ void __launch_bounds__(Shape<D, KERNEL>::kThreads, Shape<D, KERNEL>::kPerSm)
    paged_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const PagedDev p) {
    using Kernel = Shape<D, KERNEL>;
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
    locate<Kernel::kTiles, Kernel::kThreads>(p, bar);
    __syncthreads();
    if constexpr (KERNEL == kMixed) {
        if (bar.pair)
            work<D, F16, 2, KERNEL>(tm_q, tm_k, tm_v, p, smem, bar);
        else
            work<D, F16, 1, KERNEL>(tm_q, tm_k, tm_v, p, smem, bar);
    } else {
        work<D, F16, 1, KERNEL>(tm_q, tm_k, tm_v, p, smem, bar);
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

Plan plan_of(const attn_paged_params& p, int num_sms) {
    const int G = p.num_q_heads / p.num_kv_heads;
    Plan pl;
    pl.tiles = (long long)p.max_q * G > BM ? 2 : 1;
    pl.num_sms = num_sms;
    pl.tok_tile = BM / G;
    if (pl.tiles == 1 && p.max_q < pl.tok_tile) pl.tok_tile = p.max_q;
    pl.rows = pl.tok_tile * G;
    const bool few = p.d == 128 && pl.rows <= kFewRows && (long long)p.max_pages * p.page_size <= kFewKeys;
    pl.kernel = pl.tiles == 2 ? kMixed : few ? kFew : kOne;
    pl.ctas = num_sms * (pl.kernel == kFew || (pl.kernel == kOne && p.d == 64) ? 2 : 1);  // Shape::kPerSm
    // the workspace has room for either one-tile kernel, so that its size does not go by the table's
    const int room = num_sms * (pl.tiles == 1 && (p.d == 64 || pl.rows <= kFewRows) ? 2 : 1);
    pl.meta_bytes = ((size_t)room * 2 * sizeof(int4) + 255) / 256 * 256;
    pl.bytes = pl.meta_bytes + (size_t)room * 2 * pl.tiles * pl.rows * (p.d + 4) * sizeof(float);
    return pl;
}

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

template <int D, bool F16, int KERNEL>
cudaError_t launch_tc(const CUtensorMap (&maps)[3], const PagedDev& p, int grid, cudaStream_t s) {
    using Kernel = Shape<D, KERNEL>;
    const cudaError_t e = cudaFuncSetAttribute(paged_tc_kernel<D, F16, KERNEL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Kernel::kSmemBytes);
    if (e != cudaSuccess) return e;
    return launch_pdl(paged_tc_kernel<D, F16, KERNEL>, dim3(grid), dim3(Kernel::kThreads), Kernel::kSmemBytes, s, maps[0],
                      maps[1], maps[2], p);
}

// Held from a call's first launch to its last, so that calls of several host threads on one stream may share
// a workspace: the parts that one call leaves there are merged before the next call's are written.
std::mutex g_launch_mu;

template <int D, bool F16>
cudaError_t launch_both(const CUtensorMap (&maps)[3], const PagedDev& p, const Plan& pl, int grid, cudaStream_t s) {
    std::lock_guard<std::mutex> lock(g_launch_mu);
    cudaError_t e;
    if (pl.kernel == kMixed) {
        e = launch_tc<D, F16, kMixed>(maps, p, grid, s);
    } else if (D == 128 && pl.kernel == kFew) {
        e = launch_tc<128, F16, kFew>(maps, p, grid, s);
    } else {
        e = launch_tc<D, F16, kOne>(maps, p, grid, s);
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

}  // namespace

size_t paged_workspace_bytes(const attn_paged_params& p, int num_sms) { return plan_of(p, num_sms).bytes; }

attn_status_t launch_paged(const attn_paged_params& p, const LaunchCommon& lc, cudaStream_t s) {
    PFN_cuTensorMapEncodeTiled_v12000 enc;
    const attn_status_t st = map_encoder(&enc);
    if (st != ATTN_OK) return st;
    const Plan pl = plan_of(p, lc.num_sms);
    const int G = p.num_q_heads / p.num_kv_heads;
    CUtensorMap maps[3];
    // q as (column, head in the group, row, key/value head); the caches as (column, slot, head, page)
    const cuuint64_t qd[4] = {(cuuint64_t)p.d, (cuuint64_t)G, (cuuint64_t)p.total_q, (cuuint64_t)p.num_kv_heads};
    const int64_t qs[3] = {p.q_stride[1], p.q_stride[0], p.q_stride[1] * G};
    const cuuint64_t cd[4] = {(cuuint64_t)p.d, (cuuint64_t)p.page_size, (cuuint64_t)p.num_kv_heads, (cuuint64_t)p.num_pages};
    const int64_t ks[3] = {p.k_stride[2], p.k_stride[1], p.k_stride[0]}, vs[3] = {p.v_stride[2], p.v_stride[1], p.v_stride[0]};
    const cuuint32_t box_rows = (cuuint32_t)(p.page_size < BN ? p.page_size : BN);
    CUresult r = encode(enc, &maps[0], p.dtype, p.q, qd, qs, (cuuint32_t)G, (cuuint32_t)pl.tok_tile);
    if (r == CUDA_SUCCESS) r = encode(enc, &maps[1], p.dtype, p.k_cache, cd, ks, box_rows, 1);
    if (r == CUDA_SUCCESS) r = encode(enc, &maps[2], p.dtype, p.v_cache, cd, vs, box_rows, 1);
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
    a.c = p.scale * kLog2e;
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
    const bool f16 = p.dtype == ATTN_F16;
    const cudaError_t e =
        p.d == 64 ? (f16 ? launch_both<64, true>(maps, a, pl, pl.ctas, s) : launch_both<64, false>(maps, a, pl, pl.ctas, s))
                  : (f16 ? launch_both<128, true>(maps, a, pl, pl.ctas, s)
                         : launch_both<128, false>(maps, a, pl, pl.ctas, s));
    return e == cudaSuccess ? ATTN_OK : report_error(ATTN_ERR_CUDA, "attn_paged launch: %s", cudaGetErrorString(e));
}

}  // namespace attn
