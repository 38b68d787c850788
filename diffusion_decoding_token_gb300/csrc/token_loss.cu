// token_loss.cu -- log-probabilities of one given token per row, the clipped policy
// loss and the preference loss, with the gradients of all three by the logits.
//
// With q = softmax(z / T) and a the row's token, every loss here is a function of the
// rows' ln q_a, so that its gradient is slope / T ([v = a] - q_v), slope the loss's
// derivative by ln q_a (token_math.cuh has both).  `state` holds what the gradient
// needs of a row: maximum, 1 / sum, 1 - q_a, slope.
//
// The sums and the gradient are bound by HBM: one read of the row, and one write.
#include "common.cuh"
#include "launch.h"
#include "row_vec.cuh"
#include "token_math.cuh"

namespace dlm {

namespace {

constexpr int kThreads = kRowThreads;
constexpr int kWarps = kRowWarps;
constexpr float kRebase = 12.0f;  // powers of 2 of headroom before a thread's reference moves

// The sum of the weights 2^((z - ref) c), relative to the largest of them.
struct Part {
    float ref, sum;
};

__device__ __forceinline__ float or_zero(float ref) { return ref > -INFINITY ? ref : 0.f; }
__device__ __forceinline__ Part merge(Part a, Part b, float c) {
    const float ref = max_nan(a.ref, b.ref), to = or_zero(ref);
    return Part{ref, a.sum * ex2((a.ref - to) * c) + b.sum * ex2((b.ref - to) * c)};
}
__device__ __forceinline__ Part warp_merge(Part a, float c) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
        a = merge(a, Part{__shfl_xor_sync(DLM_FULL_MASK, a.ref, o), __shfl_xor_sync(DLM_FULL_MASK, a.sum, o)}, c);
    return a;
}

// Element e of a vector replaced by the bits x.
template <int DT>
__device__ __forceinline__ uint4 with_elem(uint4 w, int e, uint32_t x) {
    uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == DLM_F32) {
            if (i == e) r[i] = x;
        } else {
            if (i == e >> 1) r[i] = e & 1 ? (r[i] & 0xffffu) | x << 16 : (r[i] & 0xffff0000u) | x;
        }
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}
template <int DT>
__device__ constexpr uint32_t neg_inf_bits() {
    if constexpr (DT == DLM_F32)
        return 0xff800000u;
    else
        return Row<DT>::kNegInf;
}
template <int DT>
__device__ __forceinline__ uint32_t elem_bits(float x) {
    if constexpr (DT == DLM_F32) {
        return __float_as_uint(x);
    } else if constexpr (DT == DLM_BF16) {
        return __bfloat16_as_ushort(__float2bfloat16_rn(x));
    } else {
        return __half_as_ushort(__float2half_rn(x));
    }
}

// Adds a vector to a running sum.
template <int DT>
__device__ __forceinline__ void add_vector(Part& p, uint4 w, float c, float c_lo) {
    constexpr int EPV = Row<DT>::EPV;
    const float m = Row<DT>::vmax(w);
    if (!((m - p.ref) * c <= kRebase)) {  // (NaN moves it too)
        p.sum *= ex2((p.ref - or_zero(m)) * c);
        p.ref = m;
    }
    float z[EPV];
    Row<DT>::unpack(w, z);
    const float ref = or_zero(p.ref);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < EPV; ++i) s += ex2(fmaf(z[i] - ref, c, (z[i] - ref) * c_lo));
    p.sum += s;
}

// A vector of a row that the kernel may also write.
template <int DT>
__device__ __forceinline__ uint4 load_row(const char* row, int64_t V, int v) {
    return (int64_t)(v + 1) * Row<DT>::EPV <= V ? ld_row(reinterpret_cast<const uint4*>(row) + v) : load_vec<DT>(row, V, v);
}

// What a row's loss is, by the thread that has its sums: its slope.
__device__ float finish_row(const TokenArgs& a, int64_t o, const TokenRow& t, float weight) {
    if (!t.ok) raise_status(a.dev_status, DLM_DEV_NONFINITE);
    LossSlope x{0.f, weight};
    double term = 0.0;
    if (a.op == kTokenPolicy) {
        x = policy_row(a.policy, t.logp, weight, a.advantages[o], a.old_logp != nullptr, a.old_logp ? a.old_logp[o] : 0.f,
                       a.ref_logp ? a.ref_logp[o] : 0.f);
        a.loss[o] = x.loss;
        if (t.ok && x.slope != x.slope) raise_status(a.dev_status, DLM_DEV_NONFINITE);
    } else if (a.op == kTokenPreference) {
        term = (double)weight * (t.logp - (a.ref_logp ? (double)a.ref_logp[o] : 0.0));
    }
    if (a.logp) a.logp[o] = (float)t.logp;
    if (a.lse) a.lse[o] = (float)t.lse;
    if (a.state) {
        float* s = a.state + o * DLM_TOKEN_STATE;
        s[0] = t.m;
        s[1] = t.inv;
        s[2] = t.away;
        s[3] = a.op == kTokenPreference ? 0.f : x.slope;  // a row in no pair: 0
        *reinterpret_cast<double*>(s + 4) = term;
        s[6] = __int_as_float(-1);
        s[7] = 0.f;
    }
    return x.slope;
}
// A row without a loss.
__device__ void finish_none(const TokenArgs& a, int64_t o) {
    if (a.op == kTokenPolicy) a.loss[o] = 0.f;
    if (a.logp) a.logp[o] = 0.f;
    if (a.lse) a.lse[o] = 0.f;
    if (a.state) {
        float4* s = reinterpret_cast<float4*>(a.state + o * DLM_TOKEN_STATE);
        s[0] = make_float4(0.f, 0.f, 0.f, 0.f);
        s[1] = make_float4(0.f, 0.f, __int_as_float(-1), 0.f);
    }
}

// SUMS: the row's sums and what follows from them; GRAD: its gradient, from the sums
// or from the state.
template <int DT, bool SUMS, bool GRAD>
__global__ void __launch_bounds__(kThreads) token_row_kernel(const TokenArgs a) {
    constexpr int EPV = Row<DT>::EPV;
    __shared__ Part s_part[kWarps];
    __shared__ float4 s_row;
    const int t = threadIdx.x;
    const int64_t r = blockIdx.x, V = a.vocab;
    int64_t q = r;
    if (SUMS && a.row_index) {
        q = a.row_index[r];
        if (q < 0 || (a.n_src > 0 && q >= a.n_src)) {
            if (t == 0) raise_status(a.dev_status, DLM_DEV_BAD_INDEX);
            return;
        }
    }
    const int64_t o = a.gather ? r : q;
    const int token = a.tokens[o];
    const char* row = static_cast<const char*>(a.logits) + q * a.row_stride * Row<DT>::ESZ;
    const int nv = (int)((V + EPV - 1) / EPV);
    bool none = token < 0 || token >= V;
    float m = 0.f, inv = 0.f, away = 0.f, k = 0.f;
    if (SUMS) {
        const float weight = a.weights ? a.weights[o] : 1.f;
        none = none || weight == 0.f;
        if (none) {
            if (t == 0) {
                if (token >= V) raise_status(a.dev_status, DLM_DEV_BAD_INDEX);
                finish_none(a, o);
            }
        } else {
            Part p{-FLT_MAX, 0.f};
            for (int v = t; v < nv; v += kThreads) {
                uint4 w = load_row<DT>(row, V, v);
                if (v == token / EPV) w = with_elem<DT>(w, token % EPV, neg_inf_bits<DT>());
                add_vector<DT>(p, w, a.scale, a.scale_lo);
            }
            p = warp_merge(p, a.scale);
            if ((t & 31) == 0) s_part[t >> 5] = p;
            __syncthreads();
            if (t == 0) {
                for (int i = 1; i < kWarps; ++i) p = merge(p, s_part[i], a.scale);
                const float z = Row<DT>::scalar(row, token), top = max_nan(p.ref, z);
                const TokenRow x = token_row(p.ref, p.sum, z, ex2((z - top) * a.scale), ex2((p.ref - top) * a.scale), a.inv_t);
                s_row = make_float4(x.m, x.inv, x.away, finish_row(a, o, x, weight));
            }
            __syncthreads();
            m = s_row.x;
            inv = s_row.y;
            away = s_row.z;
            k = s_row.w * (float)a.inv_t;
        }
    } else {
        const float* s = a.state + r * DLM_TOKEN_STATE;
        m = s[0];
        inv = s[1];
        away = s[2];
        k = s[3] * (float)a.inv_t;
        if (a.grad_loss) {
            const int64_t at = a.op == kTokenPreference ? (int64_t)__float_as_int(s[6]) : r;
            k *= at >= 0 && at < a.n_up ? a.grad_loss[at] : 0.f;
        }
    }
    if (!GRAD) return;
    none = none || k == 0.f || inv == 0.f;
    char* out = static_cast<char*>(a.grad) + r * a.grad_stride * Row<DT>::ESZ;
    for (int v = t; v < nv; v += kThreads) {
        uint32_t g[EPV];
        if (none) {
#pragma unroll
            for (int e = 0; e < EPV; ++e) g[e] = 0;
        } else {
            float z[EPV];
            Row<DT>::unpack(load_row<DT>(row, V, v), z);
#pragma unroll
            for (int e = 0; e < EPV; ++e)
                g[e] = elem_bits<DT>(v * EPV + e == token ? k * away : -k * inv * ex2((z[e] - m) * a.scale));
        }
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
            if ((int64_t)v * EPV + e >= V) break;
            if constexpr (DT == DLM_F32)
                reinterpret_cast<uint32_t*>(out)[(int64_t)v * EPV + e] = g[e];
            else
                reinterpret_cast<uint16_t*>(out)[(int64_t)v * EPV + e] = (uint16_t)g[e];
        }
    }
}

// The offsets' bounds [b, e) of sequence s as they should be: within the rows and in
// order (each offset at least its predecessors).
__device__ __forceinline__ int64_t clean_offset(const TokenArgs& a, int64_t s) {
    int64_t most = 0;
    for (int64_t i = threadIdx.x & 31; i <= s; i += 32) most = max(most, (int64_t)a.offsets[i]);
#pragma unroll
    for (int o = 16; o; o >>= 1) most = max(most, __shfl_xor_sync(DLM_FULL_MASK, most, o));
    return min(most, a.n_rows);
}

// One CTA per pair: the scores, the loss, and the slope of every row of the pair.
__global__ void __launch_bounds__(kThreads) pair_kernel(const TokenArgs a) {
    __shared__ double s_sum[2][kWarps];
    __shared__ float s_slope;
    const int t = threadIdx.x;
    const int64_t i = blockIdx.x;
    int64_t at[3];
    for (int j = 0; j < 3; ++j) {
        at[j] = clean_offset(a, 2 * i + j);
        if (t == 0 && at[j] != a.offsets[2 * i + j]) raise_status(a.dev_status, DLM_DEV_BAD_INDEX);
    }
    for (int side = 0; side < 2; ++side) {
        double sum = 0.0;
        for (int64_t r = at[side] + t; r < at[side + 1]; r += kThreads)
            sum += *reinterpret_cast<const double*>(a.state + r * DLM_TOKEN_STATE + 4);
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(DLM_FULL_MASK, sum, o);
        if ((t & 31) == 0) s_sum[side][t >> 5] = sum;
    }
    __syncthreads();
    if (t == 0) {
        double score[2];
        for (int side = 0; side < 2; ++side) {
            score[side] = 0.0;
            for (int w = 0; w < kWarps; ++w) score[side] += s_sum[side][w];
            if (a.score) a.score[2 * i + side] = (float)score[side];
        }
        const LossSlope x = preference_pair(a.preference, score[0], score[1], a.margins ? a.margins[i] : 0.f,
                                            a.pair_weights ? a.pair_weights[i] : 1.f);
        a.loss[i] = x.loss;
        s_slope = x.slope;
        if (x.slope != x.slope) raise_status(a.dev_status, DLM_DEV_NONFINITE);
    }
    __syncthreads();
    for (int side = 0; side < 2; ++side)
        for (int64_t r = at[side] + t; r < at[side + 1]; r += kThreads) {
            float* s = a.state + r * DLM_TOKEN_STATE;
            if (s[1] == 0.f) continue;  // no loss of its own
            s[3] = (side ? -s_slope : s_slope) * (a.weights ? a.weights[r] : 1.f);
            s[6] = __int_as_float((int)i);
        }
}

}  // namespace

size_t preference_workspace(int64_t n_rows, int64_t n_pairs) {
    (void)n_pairs;
    return (size_t)(n_rows * DLM_TOKEN_STATE * 4 + 16);
}

template <int DT>
static cudaError_t run_token(TokenArgs a, cudaStream_t st) {
    if (a.workspace) a.state = static_cast<float*>(a.workspace);
    const unsigned n = (unsigned)a.n_rows;
    if (a.op == kTokenPreference && a.sums) {
        if (n) token_row_kernel<DT, true, false><<<n, kThreads, 0, st>>>(a);
        if (a.n_pairs > 0) pair_kernel<<<(unsigned)a.n_pairs, kThreads, 0, st>>>(a);
        if (a.grad && n) token_row_kernel<DT, false, true><<<n, kThreads, 0, st>>>(a);
    } else if (!a.sums) {
        token_row_kernel<DT, false, true><<<n, kThreads, 0, st>>>(a);
    } else if (!a.grad) {
        token_row_kernel<DT, true, false><<<n, kThreads, 0, st>>>(a);
    } else {
        token_row_kernel<DT, true, true><<<n, kThreads, 0, st>>>(a);
    }
    return cudaGetLastError();
}

cudaError_t launch_token(const TokenArgs& a, int dtype, cudaStream_t st) {
    switch (dtype) {
    case DLM_BF16: return run_token<DLM_BF16>(a, st);
    case DLM_F16: return run_token<DLM_F16>(a, st);
    default: return run_token<DLM_F32>(a, st);
    }
}

}  // namespace dlm
