// row_vec.cuh -- reading vocab-wide rows in 16-byte vectors, and block-wide
// sums, shared by the row search and the distillation kernels.
#pragma once

#include <cooperative_groups.h>
#include <float.h>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace dlm {

namespace {

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;

__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
    uint4 r;
    asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
        : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
        : "l"(p));
    return r;
}

// The same without the read-only path: for rows that the kernel also writes.
__device__ __forceinline__ uint4 ld_row(const uint4* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}
__device__ __forceinline__ void st_row(uint4* p, uint4 v) {
    asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}

// Maximum over the warp, NaN if any lane holds one.
__device__ __forceinline__ float warp_max_nan(float v) {
    float m;
    asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}

template <int DT>
struct Row;

template <>
struct Row<DLM_BF16> {
    static constexpr int EPV = 8, ESZ = 2;
    static constexpr uint32_t kNegInf = 0xff80u;
    static __device__ __forceinline__ void unpack(uint4 w, float (&z)[8]) {
        const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            z[2 * i] = __uint_as_float(r[i] << 16);
            z[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ float vmax(uint4 w) {
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&w);
        const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
        return max_nan(__low2float(m), __high2float(m));
    }
    static __device__ __forceinline__ float scalar(const void* p, int64_t i) {
        return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
    }
};

template <>
struct Row<DLM_F16> {
    static constexpr int EPV = 8, ESZ = 2;
    static constexpr uint32_t kNegInf = 0xfc00u;
    static __device__ __forceinline__ void unpack(uint4 w, float (&z)[8]) {
        const __half2* h = reinterpret_cast<const __half2*>(&w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(h[i]);
            z[2 * i] = f.x;
            z[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ float vmax(uint4 w) {
        const __half2* h = reinterpret_cast<const __half2*>(&w);
        const __half2 m = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
        return max_nan(__low2float(m), __high2float(m));
    }
    static __device__ __forceinline__ float scalar(const void* p, int64_t i) {
        return __half2float(static_cast<const __half*>(p)[i]);
    }
};

template <>
struct Row<DLM_F32> {
    static constexpr int EPV = 4, ESZ = 4;
    static __device__ __forceinline__ void unpack(uint4 w, float (&z)[4]) {
        z[0] = __uint_as_float(w.x);
        z[1] = __uint_as_float(w.y);
        z[2] = __uint_as_float(w.z);
        z[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ float vmax(uint4 w) {
        return max_nan(max_nan(__uint_as_float(w.x), __uint_as_float(w.y)),
                       max_nan(__uint_as_float(w.z), __uint_as_float(w.w)));
    }
    static __device__ __forceinline__ float scalar(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
};

// Vector v of a row of V elements; elements at or past V read as -inf (the
// row's last vector is read element by element when V cuts it, so nothing
// past the row is touched).
template <int DT>
__device__ __forceinline__ uint4 load_vec(const char* row, int64_t V, int v) {
    constexpr int EPV = Row<DT>::EPV;
    if ((int64_t)(v + 1) * EPV <= V) return ld_stream(reinterpret_cast<const uint4*>(row) + v);
    uint32_t w[4];
    if constexpr (DT == DLM_F32) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t i = (int64_t)v * EPV + e;
            w[e] = i < V ? reinterpret_cast<const uint32_t*>(row)[i] : 0xff800000u;
        }
    } else {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t i = (int64_t)v * EPV + 2 * e;
            const uint32_t lo = i < V ? p[i] : Row<DT>::kNegInf, hi = i + 1 < V ? p[i + 1] : Row<DT>::kNegInf;
            w[e] = lo | (hi << 16);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// ---- block-wide helpers (every thread of the CTA calls them) --------------

// Exclusive sum over the threads; `total` is the sum over all of them.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* scratch, uint64_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(DLM_FULL_MASK, inc, o);
        if (lane >= o) inc += x;
    }
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    uint64_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) {
        if (w < warp) before += scratch[w];
        total += scratch[w];
    }
    __syncthreads();
    return before + inc - v;
}

__device__ __forceinline__ float block_max_nan(float v, float* scratch) {
    v = warp_max_nan(v);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    float m = scratch[0];
#pragma unroll
    for (int w = 1; w < kRowWarps; ++w) m = max_nan(m, scratch[w]);
    __syncthreads();
    return m;
}

// The CTAs that work one row (rank 0 merges).  With one CTA the cluster
// barrier is the block's.
struct Cluster {
    int split, rank;
    __device__ void sync() const {
        if (split > 1)
            cg::this_cluster().sync();
        else
            __syncthreads();
    }
    template <typename T>
    __device__ T* at(T* p, int r) const {
        return split > 1 ? cg::this_cluster().map_shared_rank(p, r) : p;
    }
};

}  // namespace

}  // namespace dlm
