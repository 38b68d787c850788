// distill.cu -- distillation of a student's logit rows from the teacher's top
// logits: the loss of a row, its gradient, or both in one launch.
//
// With q = softmax(s / T) over the student's row s and p the teacher's
// probabilities of the listed ids (softmax(t / T) over the list, or
// exp(t / T - lse_t) with p_rest = 1 - sum p for every other token together):
//   loss   = w [ sum_j p_j (ln p_j - ln q_{id_j}) + p_rest (ln p_rest - ln q_rest) ]
//   dl/ds_v = w / T (q_v - p_v)                  v listed (p_v: all its entries)
//   dl/ds_v = w / T q_v (1 - p_rest / q_rest)    otherwise (p_rest = 0: w / T q_v)
// Everything the gradient needs of a row is its maximum, 1 / sum, the factor
// of the tokens that are not listed, and the list: `state` holds it between
// the two calls.
//
// The loss reads the row once (HBM-bound).  q_rest = 1 - sum q_id would lose
// all digits for a peaked student, so the sum over the tokens that are not
// listed is taken apart from the start: a bitmap of the CTA's slice in shared
// memory marks the listed ones, and one byte of it answers for a whole vector.
// The gradient is written for every token as if none were listed, and then the
// listed ones are written over (the block barrier between orders the two).
#include "common.cuh"
#include "launch.h"
#include "row_vec.cuh"
#include "weight.cuh"

namespace dlm {

namespace {

constexpr int kThreads = kRowThreads;
constexpr int kWarps = kRowWarps;
constexpr int kUnroll = 4;
constexpr float kRebase = 12.0f;  // powers of 2 of headroom before a thread's reference moves
constexpr float kUnit = 5.684341886080802e-14f;  // 2^-44

// A slice's softmax sums relative to `ref`; `mx` is the exact maximum (NaN if
// the slice holds one), `rest` the sum over the tokens that are not listed.
struct Sums {
    float mx, ref, all, rest;
};

__device__ __forceinline__ void merge(Sums& a, const Sums& b, float c) {
    const float r = fmaxf(a.ref, b.ref);
    const float ea = ex2((a.ref - r) * c), eb = ex2((b.ref - r) * c);
    a.all = a.all * ea + b.all * eb;
    a.rest = a.rest * ea + b.rest * eb;
    a.ref = r;
    a.mx = max_nan(a.mx, b.mx);
}

// Merge over the warp in a fixed order (lower lane first), all lanes agree.
__device__ __forceinline__ void warp_merge(Sums& a, float c) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        Sums b;
        b.mx = __shfl_xor_sync(DLM_FULL_MASK, a.mx, o);
        b.ref = __shfl_xor_sync(DLM_FULL_MASK, a.ref, o);
        b.all = __shfl_xor_sync(DLM_FULL_MASK, a.all, o);
        b.rest = __shfl_xor_sync(DLM_FULL_MASK, a.rest, o);
        if (threadIdx.x & o) {
            merge(b, a, c);
            a = b;
        } else {
            merge(a, b, c);
        }
    }
}

struct Shared {
    Sums warp[kWarps];
    Sums cta;
    Sums row;
    uint64_t scan[kWarps];
    float fscan[kWarps];
    double dscan[kWarps];
    float m, inv, tail;       // the row's state
    float p_rest;
    int any;                  // listed entries in range
    int bad;                  // a teacher logit was NaN or +inf
    int repeated;             // an id is listed more than once
};

// The list in shared memory.
struct List {
    int32_t* id;     // -1: no entry
    float* t;        // teacher logit
    float* p;        // teacher probability
    float* s;        // student logit (entries of this CTA's slice)
    uint32_t* bits;  // the listed tokens of this CTA's slice
};

__host__ __device__ inline size_t shared_bytes() { return (sizeof(Shared) + 15) & ~(size_t)15; }

__device__ __forceinline__ List carve(unsigned char* p, int k) {
    List l;
    p += shared_bytes();
    l.id = reinterpret_cast<int32_t*>(p);
    l.t = reinterpret_cast<float*>(l.id + k);
    l.p = l.t + k;
    l.s = l.p + k;
    l.bits = reinterpret_cast<uint32_t*>(l.s + k);
    return l;
}

__device__ __forceinline__ float teacher_at(const DistillArgs& a, int64_t i) {
    switch (a.teacher_dtype) {
    case DLM_BF16: return Row<DLM_BF16>::scalar(a.teacher, i);
    case DLM_F16: return Row<DLM_F16>::scalar(a.teacher, i);
    default: return static_cast<const float*>(a.teacher)[i];
    }
}

__device__ __forceinline__ double block_sum(double v, double* scratch) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(DLM_FULL_MASK, v, o);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    double s = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += scratch[w];
    __syncthreads();
    return s;
}

// Reads the row's list and turns the teacher's logits into probabilities.
// lse_t is used when rest.  Returns the natural log of the teacher's
// normaliser (t / T - log_z = ln p).
__device__ double read_list(const DistillArgs& a, const List& l, Shared& sh, int64_t r, bool rest, float lse_t) {
    const int t = threadIdx.x, K = a.k;
    float mx = -INFINITY;
    bool any = false, bad = false;
    for (int j = t; j < K; j += kThreads) {
        int id = a.ids[r * K + j];
        if (id >= a.vocab) {
            id = -1;
            raise_status(a.dev_status, DLM_DEV_BAD_INDEX);
        }
        const float x = teacher_at(a, r * K + j);
        if (id >= 0) {
            any = true;
            bad |= !(x < INFINITY);  // +inf or NaN
            mx = fmaxf(mx, x);
        }
        l.id[j] = id < 0 ? -1 : id;
        l.t[j] = x;
    }
    if (rest) bad |= !(fabsf(lse_t) < INFINITY);
    mx = block_max_nan(mx, sh.fscan);
    any = __syncthreads_or(any);
    bad = __syncthreads_or(bad);
    const double inv_t = 1.0 / (double)a.temperature;
    const bool none = mx == -INFINITY;  // no entry, or only such that carry nothing
    const WeightScale ws = weight_scale(none ? 0.f : mx, a.temperature);
    uint64_t sum = 0;
    for (int j = t; j < K; j += kThreads) {
        float p = 0.f;
        if (l.id[j] >= 0) {
            // p (before the renormalisation) = 2^-(y + lo); the integer weight
            // serves the sum, which p_rest is the difference of 1 and, and the
            // float keeps all its digits for a small p
            float y, lo;
            if (rest) {
                // a lse_t below the logits (p above 1) counts as p = 1
                const double d = fmax(0.0, ((double)lse_t - (double)l.t[j] * inv_t) * 1.4426950408889634);
                y = (float)d;
                lo = y < INFINITY ? (float)(d - (double)y) : 0.f;
            } else {
                y = weight_exponent(l.t[j], ws, lo);
            }
            sum += weight44_of(y, lo);
            p = y < INFINITY ? exp2f(-y) * fmaf(lo, -kLn2, 1.0f) : 0.f;
        }
        l.p[j] = p;
    }
    uint64_t total;
    block_scan(sum, sh.scan, total);
    double log_z = lse_t;
    if (!rest) {
        const float inv = total ? 1.0f / ((float)total * kUnit) : 0.f;
        for (int j = t; j < K; j += kThreads) l.p[j] *= inv;
        log_z = (double)mx * inv_t + log((double)total * (double)kUnit);
    }
    if (t == 0) {
        sh.any = any && !none;
        sh.bad = bad;
        const uint64_t one = 1ull << kWeightBits;
        sh.p_rest = rest && total < one ? (float)(one - total) * kUnit : 0.f;
    }
    __syncthreads();
    return log_z;
}

// Sums of vectors [v0, v1) of a row (kThreads threads; the whole CTA calls).
template <int DT, bool REST>
__device__ Sums stream_sums(const char* row, int64_t V, int v0, int v1, float c, const uint32_t* bits) {
    constexpr int EPV = Row<DT>::EPV;
    Sums a;
    a.mx = -INFINITY;
    a.ref = -FLT_MAX;
    f2 all = pack2(0.f, 0.f), rest = pack2(0.f, 0.f);
    const f2 c2 = pack2(c, c);
    const int whole = (int)min((int64_t)v1, V / EPV);
    auto add = [&](uint4 w, int v) {
        const float m = Row<DT>::vmax(w);
        a.mx = max_nan(a.mx, m);
        if ((m - a.ref) * c > kRebase) {
            const float e = ex2((a.ref - m) * c);
            all = mul2(all, pack2(e, e));
            rest = mul2(rest, pack2(e, e));
            a.ref = m;
        }
        float z[EPV];
        Row<DT>::unpack(w, z);
        const f2 r2 = pack2(a.ref, a.ref);
        f2 e[EPV / 2];
#pragma unroll
        for (int p = 0; p < EPV / 2; ++p) e[p] = ex2x2(mul2(sub2(pack2(z[2 * p], z[2 * p + 1]), r2), c2));
        if (REST) {
            const int at = (v - v0) * EPV;  // first token of the vector, from the slice's start
            const uint32_t in = (bits[at >> 5] >> (at & 31)) & ((1u << EPV) - 1u);
            if (in) {
#pragma unroll
                for (int p = 0; p < EPV / 2; ++p) {
                    float x, y;
                    unpack2(e[p], x, y);
                    const float lx = (in >> (2 * p)) & 1u ? x : 0.f, ly = (in >> (2 * p + 1)) & 1u ? y : 0.f;
                    all = add2(all, pack2(lx, ly));
                    rest = add2(rest, pack2(x - lx, y - ly));
                }
                return;
            }
        }
#pragma unroll
        for (int h = EPV / 4; h; h >>= 1)
#pragma unroll
            for (int p = 0; p < h; ++p) e[p] = add2(e[p], e[p + h]);
        rest = add2(rest, e[0]);
    };
    int v = v0 + (int)threadIdx.x;
    const uint4* vec = reinterpret_cast<const uint4*>(row);
    for (; v + (kUnroll - 1) * kThreads < whole; v += kUnroll * kThreads) {
        uint4 w[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) w[u] = ld_row(vec + v + u * kThreads);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) add(w[u], v + u * kThreads);
    }
    for (; v < v1; v += kThreads) add(v < whole ? ld_row(vec + v) : load_vec<DT>(row, V, v), v);
    a.rest = hsum2(rest);
    a.all = hsum2(all) + a.rest;  // `all` held the listed ones so far
    return a;
}

// The row's sums over all the CTAs of its cluster, in every CTA.
__device__ Sums merge_row(const Cluster& cl, Shared& sh, Sums a, float c) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    warp_merge(a, c);
    if (lane == 0) sh.warp[warp] = a;
    __syncthreads();
    if (warp == 0) {
        a = lane < kWarps ? sh.warp[lane] : Sums{-INFINITY, -FLT_MAX, 0.f, 0.f};
        warp_merge(a, c);
        if (lane == 0) sh.cta = a;
    }
    cl.sync();
    if (warp == 0) {
        a = lane < cl.split ? *cl.at(&sh.cta, lane) : Sums{-INFINITY, -FLT_MAX, 0.f, 0.f};
        warp_merge(a, c);
        if (lane == 0) sh.row = a;
    }
    cl.sync();
    return sh.row;
}

// One float to storage.
template <int DT>
__device__ __forceinline__ void store_elem(void* row, int64_t i, float x) {
    if constexpr (DT == DLM_F32)
        static_cast<float*>(row)[i] = x;
    else if constexpr (DT == DLM_BF16)
        static_cast<__nv_bfloat16*>(row)[i] = __float2bfloat16_rn(x);
    else
        static_cast<__half*>(row)[i] = __float2half_rn(x);
}

template <int DT>
__device__ __forceinline__ uint4 pack(const float (&x)[Row<DT>::EPV]) {
    uint4 w;
    uint32_t* r = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == DLM_F32) {
            r[i] = __float_as_uint(x[i]);
        } else if constexpr (DT == DLM_BF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            r[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            r[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    return w;
}

// scale * 2^((z - m) c) for vectors [v0, v1) of the row; scale = 0 writes
// zeros without reading.  In place is fine: a vector is read before it is
// written, by the same thread.
template <int DT>
__device__ void stream_grad(const char* row, char* out, int64_t V, int v0, int v1, float m, float c, float scale) {
    constexpr int EPV = Row<DT>::EPV;
    const int whole = (int)min((int64_t)v1, V / EPV);
    auto value = [&](uint4 w) {
        float z[EPV];
        Row<DT>::unpack(w, z);
#pragma unroll
        for (int e = 0; e < EPV; ++e) z[e] = scale * ex2((z[e] - m) * c);
        return pack<DT>(z);
    };
    const uint4* src = reinterpret_cast<const uint4*>(row);
    uint4* dst = reinterpret_cast<uint4*>(out);
    int v = v0 + (int)threadIdx.x;
    if (scale == 0.f) {
        for (; v < whole; v += kThreads) st_row(dst + v, make_uint4(0, 0, 0, 0));
    } else {
        for (; v + (kUnroll - 1) * kThreads < whole; v += kUnroll * kThreads) {
            uint4 w[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) w[u] = ld_row(src + v + u * kThreads);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) st_row(dst + v + u * kThreads, value(w[u]));
        }
        for (; v < whole; v += kThreads) st_row(dst + v, value(ld_row(src + v)));
    }
    if (v1 > whole) {  // the row's last, cut vector
        for (int64_t i = (int64_t)whole * EPV + threadIdx.x; i < V; i += kThreads)
            store_elem<DT>(out, i, scale == 0.f ? 0.f : scale * ex2((Row<DT>::scalar(row, i) - m) * c));
    }
}

// The listed tokens of this CTA's slice [e0, e1): g (q_v - p_v), once per
// token (the first of its entries writes, p_v adds up all of them).
template <int DT>
__device__ void write_listed(const List& l, int K, char* out, int64_t e0, int64_t e1, float m, float c, float inv,
                             float g) {
    for (int j = threadIdx.x; j < K; j += kThreads) {
        const int id = l.id[j];
        if (id < e0 || id >= e1) continue;
        float p = 0.f;
        bool first = true;
        for (int i = 0; i < K; ++i) {
            if (l.id[i] != id) continue;
            first &= i >= j;
            p += l.p[i];
        }
        if (first) store_elem<DT>(out, id, g * (inv * ex2((l.s[j] - m) * c) - p));
    }
}

template <int DT>
struct Slice {
    int v0, v1;       // vectors of this CTA
    int64_t e0, e1;   // its tokens
    __device__ Slice(int64_t V, const Cluster& cl) {
        constexpr int EPV = Row<DT>::EPV;
        const int nv = (int)((V + EPV - 1) / EPV);
        // whole words of the bitmap per slice: 32 / EPV vectors each
        const int unit = 32 / EPV;
        const int per = ((nv + cl.split - 1) / cl.split + unit - 1) / unit * unit;
        v0 = min(nv, cl.rank * per);
        v1 = min(nv, v0 + per);
        e0 = (int64_t)v0 * EPV;
        e1 = min(V, (int64_t)v1 * EPV);
    }
};

// GRAD: the gradient in the same launch, of the sum of the row losses.
template <int DT, bool REST, bool GRAD>
__global__ void __launch_bounds__(kThreads) distill_loss_kernel(const DistillArgs a) {
    extern __shared__ __align__(16) unsigned char s_raw[];
    Shared& sh = *reinterpret_cast<Shared*>(s_raw);
    const List l = carve(s_raw, a.k);
    const int t = threadIdx.x, K = a.k;
    Cluster cl;
    cl.split = a.split;
    const int64_t r = blockIdx.x / a.split;
    cl.rank = (int)(blockIdx.x - r * a.split);
    const int64_t V = a.vocab;
    const char* row = static_cast<const char*>(a.student) + r * a.row_stride * Row<DT>::ESZ;
    char* out = GRAD ? static_cast<char*>(a.grad) + r * a.grad_stride * Row<DT>::ESZ : nullptr;
    const Slice<DT> sl(V, cl);
    const float weight = a.weights ? a.weights[r] : 1.f;
    const float c = (float)(1.4426950408889634 / (double)a.temperature);
    float* state = a.state ? a.state + r * DLM_DISTILL_STATE : nullptr;
    if (weight == 0.f) {  // the row has no loss: it is not read
        if (cl.rank == 0 && t == 0) {
            a.loss[r] = 0.f;
            if (state)
                for (int i = 0; i < DLM_DISTILL_STATE; ++i) state[i] = 0.f;
        }
        if (GRAD) stream_grad<DT>(row, out, V, sl.v0, sl.v1, 0.f, c, 0.f);
        return;
    }
    const float lse_t = REST ? a.teacher_lse[r] : 0.f;
    const double log_z = read_list(a, l, sh, r, REST, lse_t);
    if (REST) {
        const int words = (int)((sl.e1 - sl.e0 + 31) / 32);
        for (int i = t; i < words; i += kThreads) l.bits[i] = 0;
        __syncthreads();
        for (int j = t; j < K; j += kThreads) {
            const int64_t id = l.id[j];
            if (id >= sl.e0 && id < sl.e1) atomicOr(&l.bits[(id - sl.e0) >> 5], 1u << ((id - sl.e0) & 31));
        }
        __syncthreads();
    }
    const Sums q = merge_row(cl, sh, stream_sums<DT, REST>(row, V, sl.v0, sl.v1, c, l.bits), c);
    const bool fine = q.mx > -INFINITY && q.mx < INFINITY && !sh.bad;
    // sums relative to the row's maximum
    const float up = ex2((q.ref - q.mx) * c);
    const float all = q.all * up, rest = q.rest * up;
    const float p_rest = REST ? sh.p_rest : 0.f;
    const bool teaches = REST || sh.any;
    float inv = teaches ? 1.f / all : 0.f;
    float tail = REST ? (rest > 0.f ? 1.f - p_rest * (all / rest) : 0.f) : 1.f;
    if (!fine) inv = tail = NAN;
    if (cl.rank == 0) {
        const double inv_t = 1.0 / (double)a.temperature;
        const double lse_s = (double)q.mx * inv_t + log((double)all);
        double v = 0;
        for (int j = t; j < K; j += kThreads) {
            const float p = l.p[j];
            if (l.id[j] >= 0 && p > 0.f)
                v += (double)p * (((double)l.t[j] - (double)Row<DT>::scalar(row, l.id[j])) * inv_t - log_z + lse_s);
        }
        v = block_sum(v, sh.dscan);
        if (t == 0) {
            if (p_rest > 0.f) v += (double)p_rest * (log((double)p_rest) - log((double)rest / (double)all));
            if (!teaches) v = 0;
            a.loss[r] = fine ? (float)((double)weight * v) : NAN;
            if (!fine) raise_status(a.dev_status, DLM_DEV_NONFINITE);
            if (state) {
                state[0] = q.mx;
                state[1] = inv;
                state[2] = tail;
                state[3] = lse_t;
                state[4] = REST ? 1.f : 0.f;
                state[5] = state[6] = state[7] = 0.f;
            }
        }
    }
    if (GRAD) {
        for (int j = t; j < K; j += kThreads) {
            const int id = l.id[j];
            if (id >= sl.e0 && id < sl.e1) l.s[j] = Row<DT>::scalar(row, id);
        }
        cl.sync();  // in place: the first CTA has read its logits of every slice
        const float g = weight / a.temperature;
        stream_grad<DT>(row, out, V, sl.v0, sl.v1, q.mx, c, g * inv * tail);
        __syncthreads();
        if (inv != 0.f) write_listed<DT>(l, K, out, sl.e0, sl.e1, q.mx, c, inv, g);
    }
}

template <int DT>
__global__ void __launch_bounds__(kThreads) distill_grad_kernel(const DistillArgs a) {
    extern __shared__ __align__(16) unsigned char s_raw[];
    Shared& sh = *reinterpret_cast<Shared*>(s_raw);
    const List l = carve(s_raw, a.k);
    const int t = threadIdx.x, K = a.k;
    Cluster cl;
    cl.split = a.split;
    const int64_t r = blockIdx.x / a.split;
    cl.rank = (int)(blockIdx.x - r * a.split);
    const int64_t V = a.vocab;
    const char* row = static_cast<const char*>(a.student) + r * a.row_stride * Row<DT>::ESZ;
    char* out = static_cast<char*>(a.grad) + r * a.grad_stride * Row<DT>::ESZ;
    const Slice<DT> sl(V, cl);
    const float g = (a.weights ? a.weights[r] : 1.f) * (a.grad_loss ? a.grad_loss[r] : 1.f) / a.temperature;
    const float c = (float)(1.4426950408889634 / (double)a.temperature);
    const float* state = a.state + r * DLM_DISTILL_STATE;
    const float m = state[0], inv = state[1], tail = state[2];
    if (g == 0.f || inv == 0.f) {
        stream_grad<DT>(row, out, V, sl.v0, sl.v1, m, c, 0.f);
        return;
    }
    read_list(a, l, sh, r, state[4] != 0.f, state[3]);
    for (int j = t; j < K; j += kThreads) {
        const int id = l.id[j];
        if (id >= sl.e0 && id < sl.e1) l.s[j] = Row<DT>::scalar(row, id);
    }
    __syncthreads();
    stream_grad<DT>(row, out, V, sl.v0, sl.v1, m, c, g * inv * tail);
    __syncthreads();
    write_listed<DT>(l, K, out, sl.e0, sl.e1, m, c, inv, g);
}

// Shared memory of a CTA: the list, and with `bits` the bitmap of its slice.
size_t smem_bytes(int64_t V, int k, int split, bool bits) {
    size_t n = shared_bytes() + (size_t)k * 16;
    if (bits) n += (size_t)((V + split - 1) / split + 64) / 32 * 4 + 16;
    return n;
}

template <typename F>
cudaError_t launch_rows(F kernel, const DistillArgs& a, bool bits, cudaStream_t st) {
    const size_t smem = smem_bytes(a.vocab, a.k, a.split, bits);
    if (smem > 48 * 1024) {  // the same limit whatever the call's size: calls may run side by side
        const int most = (int)smem_bytes(DLM_MAX_SEARCH_VOCAB, DLM_MAX_TOPK, 1, true);
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.n_rows * a.split));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = a.split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.split > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int DT>
cudaError_t launch_loss(const DistillArgs& a, cudaStream_t st) {
    if (a.grad)
        return a.teacher_lse ? launch_rows(distill_loss_kernel<DT, true, true>, a, true, st)
                             : launch_rows(distill_loss_kernel<DT, false, true>, a, false, st);
    return a.teacher_lse ? launch_rows(distill_loss_kernel<DT, true, false>, a, true, st)
                         : launch_rows(distill_loss_kernel<DT, false, false>, a, false, st);
}

}  // namespace

// CTAs per row: a row is split over a cluster when the rows alone do not fill
// the GPU and each thread still gets a batch of vectors.
int distill_split(int dtype, int64_t n_rows, int64_t vocab, int num_sms) {
    const int64_t nv = vocab / (dtype == DLM_F32 ? 4 : 8);
    int split = 1;
    while (split < 8 && n_rows * split < 2LL * num_sms && nv / (split * 2) >= 2LL * kThreads) split *= 2;
    return split;
}

cudaError_t launch_distill_loss(const DistillArgs& a, int dtype, cudaStream_t st) {
    switch (dtype) {
    case DLM_BF16: return launch_loss<DLM_BF16>(a, st);
    case DLM_F16: return launch_loss<DLM_F16>(a, st);
    default: return launch_loss<DLM_F32>(a, st);
    }
}

cudaError_t launch_distill_grad(const DistillArgs& a, int dtype, cudaStream_t st) {
    switch (dtype) {
    case DLM_BF16: return launch_rows(distill_grad_kernel<DLM_BF16>, a, false, st);
    case DLM_F16: return launch_rows(distill_grad_kernel<DLM_F16>, a, false, st);
    default: return launch_rows(distill_grad_kernel<DLM_F32>, a, false, st);
    }
}

}  // namespace dlm
