// attn_pages_fp8.cu — keys and values stored in 8 bits in their slots, and read back.
//
// Mathematics: a row of d values becomes E4M3 codes and a power of two 2^e, the smallest with max|x| <= 448 *
// 2^e. With max|x| = m * 2^x and m in [1, 2), 448 = 1.75 * 2^8 gives e = x - 8, or x - 7 where m > 1.75: both
// are read off the bits of the maximum. x * 2^-e is exact in fp32, and the convert to E4M3 rounds to nearest
// even, so a code carries one rounding.
//
// What bounds it: a row is read and its codes written once (or the other way), so HBM; a decode step's few
// rows take a launch's latency. A lane handles 16 values of a key row and the same ones of the value row, in one
// access of 32 bytes and one of 16 each, 8 lanes (4 at d = 64) a row. Where a 16-bit row is not aligned to 32 bytes its
// access is two of 16, which touch every sector twice. 16301 rows of 8 heads with d = 128 are written in 13.8 us
// (what is written stays in L2), 65021 read back in 60.6 us (6.6 TB/s, 97 % of the measured copy rate; 67.2 with
// 16-byte accesses), a decode step's 64 rows written in 1.9 us.
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"
#include "ptx_f8.cuh"

namespace attn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kLeast = -119, kMost = 119;  // exponents of the scales

struct PagesF8Args {
    attn_pages_write_fp8_params p;
    int shift;  // log2(page_size)
    int wide;   // rows of k and v are 32-byte aligned
    int* err;
};

// (row, head) of a thread. The division is by far the dearest instruction here, in 64 bits more so.
template <int LANES>
__device__ __forceinline__ void row_head(const PagesF8Args& a, long long& row, long long& h) {
    const long long at = ((long long)blockIdx.x * (kThreads / LANES)) + threadIdx.x / LANES;
    if (at < (1ll << 32)) {
        row = (uint32_t)at / (uint32_t)a.p.num_kv_heads;
        h = (uint32_t)at % (uint32_t)a.p.num_kv_heads;
    } else {
        row = at / a.p.num_kv_heads;
        h = at % a.p.num_kv_heads;
    }
}

// Slot of a row, or -1: a row to be skipped, or a slot that the cache does not have.
__device__ __forceinline__ int slot_of(const PagesF8Args& a, long long row) {
    const int slot = a.p.slots[row];
    if (slot < 0) return -1;
    if ((slot >> a.shift) < a.p.num_pages) return slot;
    atomicCAS(a.err, 0, ATTN_ERR_INVALID);
    return -1;
}

// Exponent of the scale of a row whose largest magnitude is `top`.
__device__ __forceinline__ int exponent_of(float top) {
    const uint32_t bits = __float_as_uint(top);
    // an fp32 subnormal (exponent field 0) is below 2^kLeast * 448 like everything that kLeast stands for
    const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
    return min(max(e, kLeast), kMost);
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

template <bool F16>
struct Row16 {
    uint4 v[2];
    __device__ __forceinline__ void load(const uint16_t* src, bool wide) {
        if (wide) {
            asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                         : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[1].x), "=r"(v[1].y), "=r"(v[1].z), "=r"(v[1].w)
                         : "l"(src)
                         : "memory");
        } else {
            v[0] = *reinterpret_cast<const uint4*>(src);
            v[1] = *reinterpret_cast<const uint4*>(src + 8);
        }
    }
    __device__ __forceinline__ void get(float (&x)[16]) const {
        const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 f = ptx::unpack_h16<F16>(w[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
};

// The 16 codes of this lane; `e` is the row's exponent. LANES lanes share the row.
template <int LANES>
__device__ __forceinline__ uint4 quantise(const float (&x)[16], int& e) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[i]));  // a NaN does not count
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    e = exponent_of(top);
    const float f = pow2(-e);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = ptx_f8::pack_e4m3x4(x[4 * i] * f, x[4 * i + 1] * f, x[4 * i + 2] * f, x[4 * i + 3] * f);
    return make_uint4(c[0], c[1], c[2], c[3]);
}

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads) pages_write_fp8_kernel(const PagesF8Args a) {
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    constexpr int kLanes = D / 16;
    const attn_pages_write_fp8_params& p = a.p;
    long long row, h;
    row_head<kLanes>(a, row, h);
    const int c = (threadIdx.x % kLanes) * 16;
    const int slot = row < p.rows ? slot_of(a, row) : -1;
    Row16<F16> k{}, v{};
    if (slot >= 0) {
        k.load(static_cast<const uint16_t*>(p.k) + row * p.k_row_stride[0] + h * p.k_row_stride[1] + c, a.wide);
        v.load(static_cast<const uint16_t*>(p.v) + row * p.v_row_stride[0] + h * p.v_row_stride[1] + c, a.wide);
    }
    float x[16];
    int ek, ev;
    k.get(x);
    const uint4 kc = quantise<kLanes>(x, ek);
    v.get(x);
    const uint4 vc = quantise<kLanes>(x, ev);
    if (slot < 0) return;
    const long long page = slot >> a.shift, off = slot & (p.page_size - 1);
    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.k_cache) + page * p.k_stride[0] + h * p.k_stride[1] + off * p.k_stride[2] + c) = kc;
    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.v_cache) + page * p.v_stride[0] + h * p.v_stride[1] + off * p.v_stride[2] + c) = vc;
    if (c == 0) {
        static_cast<uint8_t*>(p.k_scale)[page * p.k_scale_stride[0] + h * p.k_scale_stride[1] + off] = (uint8_t)(ek + 127);
        static_cast<uint8_t*>(p.v_scale)[page * p.v_scale_stride[0] + h * p.v_scale_stride[1] + off] = (uint8_t)(ev + 127);
    }
}

// 16 codes times the scale of byte s, as 16-bit values.
template <bool F16>
__device__ __forceinline__ void restore(uint16_t* dst, uint4 codes, uint32_t s, bool wide) {
    const float f = __uint_as_float(s == 0 ? 0x00400000u : s == 255 ? 0x7fc00000u : s << 23);  // E8M0: 2^-127, NaN
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
    uint32_t out[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(w[i / 2] >> (16 * (i & 1)))));
        const float2 x = ptx::unpack_h16<true>(h);
        out[i] = ptx::pack_h16<F16>(x.x * f, x.y * f);
    }
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(out[0]), "r"(out[1]), "r"(out[2]),
                     "r"(out[3]), "r"(out[4]), "r"(out[5]), "r"(out[6]), "r"(out[7])
                     : "memory");
    } else {
        *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
        *reinterpret_cast<uint4*>(dst + 8) = make_uint4(out[4], out[5], out[6], out[7]);
    }
}

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads) pages_read_fp8_kernel(const PagesF8Args a) {
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    constexpr int kLanes = D / 16;
    const attn_pages_write_fp8_params& p = a.p;
    long long row, h;
    row_head<kLanes>(a, row, h);
    const int c = (threadIdx.x % kLanes) * 16;
    const int slot = row < p.rows ? slot_of(a, row) : -1;
    if (slot < 0) return;
    const long long page = slot >> a.shift, off = slot & (p.page_size - 1);
    const uint4 kc = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.k_cache) + page * p.k_stride[0] + h * p.k_stride[1] +
                                                     off * p.k_stride[2] + c);
    const uint4 vc = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.v_cache) + page * p.v_stride[0] + h * p.v_stride[1] +
                                                     off * p.v_stride[2] + c);
    const uint32_t ks = static_cast<const uint8_t*>(p.k_scale)[page * p.k_scale_stride[0] + h * p.k_scale_stride[1] + off];
    const uint32_t vs = static_cast<const uint8_t*>(p.v_scale)[page * p.v_scale_stride[0] + h * p.v_scale_stride[1] + off];
    // the rows are this call's output
    uint16_t* k = static_cast<uint16_t*>(const_cast<void*>(p.k)) + row * p.k_row_stride[0] + h * p.k_row_stride[1] + c;
    uint16_t* v = static_cast<uint16_t*>(const_cast<void*>(p.v)) + row * p.v_row_stride[0] + h * p.v_row_stride[1] + c;
    restore<F16>(k, kc, ks, a.wide);
    restore<F16>(v, vc, vs, a.wide);
}

}  // namespace

cudaError_t launch_pages_fp8(const attn_pages_write_fp8_params& p, bool read, const LaunchCommon& lc, cudaStream_t s) {
    PagesF8Args a{};
    a.p = p;
    while ((1 << a.shift) < p.page_size) ++a.shift;
    a.err = lc.err;
    auto bits = [&](const void* base, const int64_t* st) {  // of the rows' addresses
        return reinterpret_cast<uintptr_t>(base) | (uintptr_t)(p.rows > 1 ? st[0] * 2 : 0) |
               (uintptr_t)(p.num_kv_heads > 1 ? st[1] * 2 : 0);
    };
    a.wide = ((bits(p.k, p.k_row_stride) | bits(p.v, p.v_row_stride)) & 31) == 0;
    const long long threads = (long long)p.rows * p.num_kv_heads * (p.d / 16);
    const dim3 grid((unsigned)((threads + kThreads - 1) / kThreads));
    const bool f16 = p.dtype == ATTN_F16;
    auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(kThreads), 0, s, a); };
    if (read)
        return p.d == 64 ? (f16 ? go(pages_read_fp8_kernel<64, true>) : go(pages_read_fp8_kernel<64, false>))
                         : (f16 ? go(pages_read_fp8_kernel<128, true>) : go(pages_read_fp8_kernel<128, false>));
    return p.d == 64 ? (f16 ? go(pages_write_fp8_kernel<64, true>) : go(pages_write_fp8_kernel<64, false>))
                     : (f16 ? go(pages_write_fp8_kernel<128, true>) : go(pages_write_fp8_kernel<128, false>));
}

}  // namespace attn
