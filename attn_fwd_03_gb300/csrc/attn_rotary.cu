// attn_rotary.cu — rotary positions of queries and keys, forward and backward.
//
// Mathematics: pair i of a row at position x is turned by t = x * f_i. In turns that is x * f_i / (2 pi)
// modulo 1, and only the fraction matters, so each frequency becomes a 64-bit integer F_i = f_i / (2 pi) *
// 2^64 (mod 2^64) and the angle x * F_i, a product that wraps where whole turns end. It is exact to 2^-32 of
// a turn at any 32-bit position, where fp32 angles lose 2^-24 of a position that may be a million. fp32 holds 24 of
// those 32 bits: cosine and sine are those of the upper 24, turned by the lower 8 to first order. The
// backward pass is the same turn with the sine's sign changed.
//
// What bounds it: every row is read and written once and needs 6 operations a pair, so HBM (gradients of q and k of
// 16 heads, 32768 rows and 128 columns, half of them turned side by side: 84.5 us, 6.35 TB/s, 93 % of the measured copy
// rate; 32-byte accesses where the pieces lie side by side are no faster), or latency where a step brings few rows
// (64 rows of 40 heads: 2.9 us a launch, one after another).
//
// Split: a block takes kRows rows of one batch entry and a range of heads. Its threads first make the
// block's cosines and sines (each serves every head of its row) in shared memory; a thread then keeps those
// of one row and one unit of 8 pairs in registers and goes through the heads. A unit is two 16-byte pieces
// of a 16-bit row, side by side (interleaved) or half of the rotated columns apart.
#include <cmath>
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 8;      // rows of a block, at most
constexpr int kMaxUnits = 16; // units of 16 columns in a row of 256

struct RotaryArgs {
    attn_rotary_params p;
    int units, turned;   // units of a row, and those that are rotated
    int rows, groups;    // rows of a block (a power of two); groups of `units` threads, a multiple of rows
    int heads;           // of a block's range
    int row_blocks;      // of a batch entry
    float sin_sign;
    int copy_q, copy_k;  // whether columns that are not rotated have to be copied
};

// f / (2 pi) * 2^64 modulo 2^64, for |f| < 2^32. f = m 2^e with a 24-bit m: the product of m with
// 1 / (2 pi) in 96 binary places, moved by 32 - e.
__device__ __forceinline__ uint64_t turns_of(float f) {
    const uint64_t lo96 = 0x9391054a7f09d5f4ull, hi96 = 0x28be60dbull;  // 1 / (2 pi) * 2^96
    const uint32_t bits = __float_as_uint(f), ex = (bits >> 23) & 255;
    const uint64_t m = ex ? (bits & 0x7fffff) | 0x800000 : bits & 0x7fffff;
    const int s = 182 - (int)max(ex, 1u);  // 32 - e, e = ex - 150
    const uint64_t lo = m * lo96, hi = __umul64hi(m, lo96) + m * hi96;
    uint64_t t = 0;
    if (s <= 0)
        t = lo << min(-s, 63);
    else if (s < 64)
        t = (lo >> s) | (hi << (64 - s));
    else if (s < 128)
        t = hi >> (s - 64);
    return bits >> 31 ? 0 - t : t;
}

// A unit's 16 values in fp32: a[8] of the first piece, b[8] of the second.
template <int TYPE>
struct Piece;  // 8 values as they lie in memory
template <>
struct Piece<ATTN_F32> {
    float4 lo, hi;
    __device__ __forceinline__ void load(const void* base, long long at) {
        const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
        lo = src[0];
        hi = src[1];
    }
    __device__ __forceinline__ void store(void* base, long long at) const {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
        dst[0] = lo;
        dst[1] = hi;
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = lo.x, x[1] = lo.y, x[2] = lo.z, x[3] = lo.w, x[4] = hi.x, x[5] = hi.y, x[6] = hi.z, x[7] = hi.w;
    }
    __device__ __forceinline__ void set(const float (&x)[8]) {
        lo = make_float4(x[0], x[1], x[2], x[3]);
        hi = make_float4(x[4], x[5], x[6], x[7]);
    }
};
template <bool F16>
struct Piece16 {
    uint4 v;
    __device__ __forceinline__ void load(const void* base, long long at) {
        v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
    }
    __device__ __forceinline__ void store(void* base, long long at) const {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = v;
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = ptx::unpack_h16<F16>(w[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
    __device__ __forceinline__ void set(const float (&x)[8]) {
        v = make_uint4(ptx::pack_h16<F16>(x[0], x[1]), ptx::pack_h16<F16>(x[2], x[3]), ptx::pack_h16<F16>(x[4], x[5]),
                       ptx::pack_h16<F16>(x[6], x[7]));
    }
};
template <>
struct Piece<ATTN_BF16> : Piece16<false> {};
template <>
struct Piece<ATTN_F16> : Piece16<true> {};

template <int TYPE, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a) {
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const attn_rotary_params& p = a.p;
    // of row r: 4 planes of (cos 0-3, cos 4-7, sin 0-3, sin 4-7) of the units, so that neighbouring threads
    // (units) read neighbouring 16 bytes
    __shared__ float4 s_turn[kRows][4][kMaxUnits];
    const int tid = threadIdx.x;
    const int b = blockIdx.x / a.row_blocks, row0 = (blockIdx.x % a.row_blocks) * a.rows;
    const int half = p.rotary_dim / 2;
    for (int i = tid; i < a.rows * half; i += kThreads) {
        const int r = i / half, f = i % half, n = row0 + r;
        float c = 0.f, s = 0.f;
        if (n < p.N) {
            const int x = p.positions[b * p.position_stride[0] + n * p.position_stride[1]];
            // the fraction of a turn in units of 2^-32, rounded; in units of half a turn -1 to 1
            const int t = (int)(((uint64_t)(long long)x * turns_of(p.inv_freq[f]) + 0x80000000u) >> 32);
            float s0, c0;
            sincospif((float)(t & ~0xff) * 0x1p-31f, &s0, &c0);
            const float rest = (float)(t & 0xff) * (0x1p-31f * 3.14159265f);  // radians
            c = fmaf(-s0, rest, c0);
            s = fmaf(c0, rest, s0);
        }
        float* plane = reinterpret_cast<float*>(&s_turn[r][(f >> 2) & 1][f >> 3]) + (f & 3);
        plane[0] = c * p.magnitude;
        plane[2 * kMaxUnits * 4] = s * p.magnitude * a.sin_sign;
    }
    __syncthreads();
    const int u = tid % a.units, g = tid / a.units;
    const int r = g & (a.rows - 1), n = row0 + r;
    if (g >= a.groups || n >= p.N) return;
    if (p.positions[b * p.position_stride[0] + n * p.position_stride[1]] < 0) return;
    const bool turned = u < a.turned;
    // columns of the unit's two pieces
    const int c0 = turned && !INTERLEAVED ? 8 * u : 16 * u, c1 = turned && !INTERLEAVED ? half + 8 * u : 16 * u + 8;
    float cs[8], sn[8];
    if (turned) {
        const float4 v[4] = {s_turn[r][0][u], s_turn[r][1][u], s_turn[r][2][u], s_turn[r][3][u]};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            cs[4 * i] = v[i].x, cs[4 * i + 1] = v[i].y, cs[4 * i + 2] = v[i].z, cs[4 * i + 3] = v[i].w;
            sn[4 * i] = v[2 + i].x, sn[4 * i + 1] = v[2 + i].y, sn[4 * i + 2] = v[2 + i].z, sn[4 * i + 3] = v[2 + i].w;
        }
    }
    const int step = a.groups / a.rows, last = min(p.Hq + p.Hk, (int)(blockIdx.y + 1) * a.heads);
#pragma unroll 4
    for (int h = blockIdx.y * a.heads + g / a.rows; h < last; h += step) {
        const bool is_q = h < p.Hq;
        if (!turned && !(is_q ? a.copy_q : a.copy_k)) continue;
        const int head = is_q ? h : h - p.Hq;
        const int64_t* si = is_q ? p.q_stride : p.k_stride;
        const int64_t* so = is_q ? p.q_out_stride : p.k_out_stride;
        const void* src = is_q ? p.q : p.k;
        void* dst = is_q ? p.q_out : p.k_out;
        const long long from = b * si[0] + head * si[1] + n * si[2], to = b * so[0] + head * so[1] + n * so[2];
        Piece<TYPE> x0, x1;
        x0.load(src, from + c0);
        x1.load(src, from + c1);
        if (turned) {
            float xa[8], xb[8];
            x0.get(xa);
            x1.get(xb);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (INTERLEAVED) {  // pair i: elements 2 i and 2 i + 1 of the unit's 16
                    float& e = i < 4 ? xa[2 * i] : xb[2 * i - 8];
                    float& o = i < 4 ? xa[2 * i + 1] : xb[2 * i - 7];
                    const float y0 = fmaf(e, cs[i], -(o * sn[i])), y1 = fmaf(o, cs[i], e * sn[i]);
                    e = y0;
                    o = y1;
                } else {
                    const float y0 = fmaf(xa[i], cs[i], -(xb[i] * sn[i])), y1 = fmaf(xb[i], cs[i], xa[i] * sn[i]);
                    xa[i] = y0;
                    xb[i] = y1;
                }
            }
            x0.set(xa);
            x1.set(xb);
        }
        x0.store(dst, to + c0);
        x1.store(dst, to + c1);
    }
}

template <int TYPE>
cudaError_t launch_type(const RotaryArgs& a, dim3 grid, cudaStream_t s) {
    return a.p.interleaved ? launch_pdl(rotary_kernel<TYPE, true>, grid, dim3(kThreads), 0, s, a)
                           : launch_pdl(rotary_kernel<TYPE, false>, grid, dim3(kThreads), 0, s, a);
}

// A tensor of `es`-byte elements with strides over (b, h, n); the last dimension is contiguous.
attn_status_t check_rows(const char* name, const void* ptr, const int64_t* st, const int64_t (&dims)[3], int es) {
    if (!ptr) return report_error(ATTN_ERR_INVALID, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(ptr) & 15) return report_error(ATTN_ERR_ALIGN, "%s is not 16-byte aligned", name);
    for (int i = 0; i < 3; ++i) {
        if (dims[i] <= 1) continue;
        if (st[i] <= 0)
            return report_error(ATTN_ERR_INVALID, "%s stride[%d] = %lld is not positive", name, i, (long long)st[i]);
        if (st[i] >= (1ll << 38)) return report_error(ATTN_ERR_UNSUPPORTED, "%s stride[%d] too large", name, i);
        if (st[i] * es % 16 != 0)
            return report_error(ATTN_ERR_ALIGN, "%s stride[%d] = %lld elements is not a multiple of 16 bytes", name, i,
                                (long long)st[i]);
    }
    return ATTN_OK;
}

attn_status_t rotary(const attn_rotary_params* q, bool backward, cudaStream_t s) {
    if (!q) return report_error(ATTN_ERR_INVALID, "params is NULL");
    RotaryArgs a{};
    a.p = *q;
    attn_rotary_params& p = a.p;
    if (p.B < 0 || p.N < 0 || p.Hq < 0 || p.Hk < 0)
        return report_error(ATTN_ERR_INVALID, "negative size B=%d N=%d Hq=%d Hk=%d", p.B, p.N, p.Hq, p.Hk);
    if (p.reserved0 != 0) return report_error(ATTN_ERR_INVALID, "reserved0 must be 0");
    if (p.dtype == ATTN_E4M3) return report_error(ATTN_ERR_UNSUPPORTED, "rotary positions are built for bf16, fp16 and fp32");
    if (p.dtype != ATTN_BF16 && p.dtype != ATTN_F16 && p.dtype != ATTN_F32)
        return report_error(ATTN_ERR_INVALID, "unknown dtype %d", p.dtype);
    if (p.interleaved != 0 && p.interleaved != 1)
        return report_error(ATTN_ERR_INVALID, "interleaved must be 0 or 1, got %d", p.interleaved);
    if (!std::isfinite(p.magnitude) || !(p.magnitude > 0.f))
        return report_error(ATTN_ERR_INVALID, "magnitude must be positive and finite");
    if (p.d < 1) return report_error(ATTN_ERR_INVALID, "bad head dim %d", p.d);
    if (p.d % 16 != 0 || p.d > 16 * kMaxUnits)
        return report_error(ATTN_ERR_UNSUPPORTED, "head dim %d not built (a multiple of 16, up to 256)", p.d);
    if (p.rotary_dim < 1 || p.rotary_dim > p.d)
        return report_error(ATTN_ERR_INVALID, "rotary_dim %d is not in 1 .. %d", p.rotary_dim, p.d);
    if (p.rotary_dim % 16 != 0)
        return report_error(ATTN_ERR_UNSUPPORTED, "rotary_dim %d not built (a multiple of 16)", p.rotary_dim);
    if (p.Hq > 65535 || p.Hk > 65535 || p.B > 65535)
        return report_error(ATTN_ERR_UNSUPPORTED, "B, Hq and Hk are limited to 65535");
    if (p.N > INT32_MAX - 1023) return report_error(ATTN_ERR_UNSUPPORTED, "N must not exceed 2^31 - 1024, got %d", p.N);
    if (p.B == 0 || p.N == 0 || p.Hq + p.Hk == 0) return ATTN_OK;
    if (!p.positions) return report_error(ATTN_ERR_INVALID, "positions is NULL");
    if (reinterpret_cast<uintptr_t>(p.positions) & 3) return report_error(ATTN_ERR_ALIGN, "positions is not 4-byte aligned");
    if (!p.inv_freq) return report_error(ATTN_ERR_INVALID, "inv_freq is NULL");
    if (reinterpret_cast<uintptr_t>(p.inv_freq) & 3) return report_error(ATTN_ERR_ALIGN, "inv_freq is not 4-byte aligned");
    const int64_t qd[3] = {p.B, p.Hq, p.N}, kd[3] = {p.B, p.Hk, p.N};
    const int es = p.dtype == ATTN_F32 ? 4 : 2;
    attn_status_t st;
    if (p.Hq > 0) {
        if ((st = check_rows("q", p.q, p.q_stride, qd, es)) != ATTN_OK) return st;
        if ((st = check_rows("q_out", p.q_out, p.q_out_stride, qd, es)) != ATTN_OK) return st;
    }
    if (p.Hk > 0) {
        if ((st = check_rows("k", p.k, p.k_stride, kd, es)) != ATTN_OK) return st;
        if ((st = check_rows("k_out", p.k_out, p.k_out_stride, kd, es)) != ATTN_OK) return st;
    }
    for (int i = 0; i < 2; ++i)
        if (p.position_stride[i] < 0 || p.position_stride[i] >= (1ll << 38))
            return report_error(ATTN_ERR_INVALID, "position_stride[%d] = %lld is out of range", i, (long long)p.position_stride[i]);
    auto in_place = [&](const void* x, const void* y, const int64_t* sx, const int64_t* sy, const int64_t (&dims)[3]) {
        bool same = x == y;
        for (int i = 0; i < 3; ++i) same = same && (dims[i] <= 1 || sx[i] == sy[i]);
        return same;
    };
    const bool q_in_place = in_place(p.q, p.q_out, p.q_stride, p.q_out_stride, qd);
    const bool k_in_place = in_place(p.k, p.k_out, p.k_stride, p.k_out_stride, kd);
    if ((p.Hq > 0 && p.q == p.q_out && !q_in_place) || (p.Hk > 0 && p.k == p.k_out && !k_in_place))
        return report_error(ATTN_ERR_INVALID, "an output over its input has to have its strides");
    LaunchCommon lc;
    if ((st = launch_setup(&lc)) != ATTN_OK) return st;
    a.copy_q = !q_in_place;
    a.copy_k = !k_in_place;
    a.sin_sign = backward ? -1.f : 1.f;
    a.units = p.d / 16;
    a.turned = p.rotary_dim / 16;
    a.rows = 1;
    while (a.rows < kRows && a.rows < p.N) a.rows *= 2;
    a.groups = kThreads / a.units / a.rows * a.rows;
    a.row_blocks = (p.N + a.rows - 1) / a.rows;
    const int heads = p.Hq + p.Hk, at_once = a.groups / a.rows;
    // A block takes all heads where that leaves two blocks an SM at least, else as few as its threads take at once.
    const long long blocks = (long long)p.B * a.row_blocks;
    a.heads = blocks >= 2 * lc.num_sms ? heads : at_once;
    if (blocks > INT32_MAX) return report_error(ATTN_ERR_UNSUPPORTED, "too many rows: B * N = %lld", (long long)p.B * p.N);
    const dim3 grid((unsigned)blocks, (unsigned)((heads + a.heads - 1) / a.heads));
    const cudaError_t e = p.dtype == ATTN_BF16  ? launch_type<ATTN_BF16>(a, grid, s)
                          : p.dtype == ATTN_F16 ? launch_type<ATTN_F16>(a, grid, s)
                                                : launch_type<ATTN_F32>(a, grid, s);
    return e == cudaSuccess ? ATTN_OK : report_error(ATTN_ERR_CUDA, "attn_rotary launch: %s", cudaGetErrorString(e));
}

}  // namespace
}  // namespace attn

extern "C" {

attn_status_t attn_rotary(const attn_rotary_params* p, void* stream) {
    return attn::rotary(p, false, static_cast<cudaStream_t>(stream));
}

attn_status_t attn_rotary_bwd(const attn_rotary_params* p, void* stream) {
    return attn::rotary(p, true, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
