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

constexpr int kThreads = kRowThreads;   // consumers: threads that do the arithmetic
constexpr int kWarps = kRowWarps;
constexpr int kBlock = kThreads + 64;   // and the warps that finish rows and that fetch them
constexpr int kPerThread = 2;           // vectors of a chunk per thread
constexpr int kChunkVecs = kPerThread * kThreads, kChunkBytes = kChunkVecs * 16;
constexpr int kItems = 4;               // rows that the fetching warp may be ahead
constexpr int kSlots = 8;               // rows whose shares may be on their way (more than kItems + 2)
constexpr int kMaxRing = 24;
constexpr float kRebase = 12.0f;        // powers of 2 of headroom before a thread's reference moves
constexpr long long kWaitLimit = 4000000000LL;  // ~2 s

// What a thread, a warp or a CTA knows of a row: the sum of its slice's weights
// 2^((z - ref) c), without the token's, relative to the largest logit of them; and the
// token's logit (-inf: it lies in another slice).
struct __align__(16) Part {
    float ref, sum, z, pad;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(DLM_FULL_MASK, v, o);
    return v;
}
// The sum over the lanes in a fixed order, in all lanes.
__device__ __forceinline__ Part warp_part(Part a, float c) {
    Part b;
    b.ref = warp_max_nan(a.ref);
    b.z = warp_max_nan(a.z);
    b.sum = warp_sum(a.sum * ex2((a.ref - or_zero(b.ref)) * c));
    b.pad = 0.f;
    return b;
}

// ---- barriers and copies ------------------------------------------------------

__device__ __forceinline__ void arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ uint32_t remote(const void* p, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ void arrive_at(uint64_t* bar, int rank) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote(bar, rank)) : "memory");
}
// Waits for a phase that CTAs of the cluster complete; false if that takes too long.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity) {
    long long t0 = 0;
    for (int n = 0;; ++n) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        if (n == 0)
            t0 = clock64();
        else if (clock64() - t0 > kWaitLimit)
            return false;
    }
}
// The same for a whole warp, whose lanes go on together or give up together.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity) {
    return __all_sync(DLM_FULL_MASK, wait_for(bar, parity));
}
// A share into CTA `rank`'s slot, counted there by its barrier.
__device__ __forceinline__ void send(Part* slot, uint64_t* bar, int rank, Part p) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                     remote(slot, rank)),
                 "r"(__float_as_uint(p.ref)), "r"(__float_as_uint(p.sum)), "r"(__float_as_uint(p.z)), "r"(0u),
                 "r"(remote(bar, rank))
                 : "memory");
}
// Untiled copy into this CTA's shared memory: both addresses and the size in whole 16 bytes.
__device__ __forceinline__ void fetch(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
// Asks for a cluster of the grid that has not started: its first CTA's index arrives
// in all CTAs of this one, or that there is none.
__device__ __forceinline__ void ask_next(void* answer, uint64_t* bar, bool cluster) {
    if (cluster)
        asm volatile(
            "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.multicast::cluster::all.b128 [%0], "
            "[%1];" ::"r"(smem_u32(answer)),
            "r"(smem_u32(bar))
            : "memory");
    else
        asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                         smem_u32(answer)),
                     "r"(smem_u32(bar))
                     : "memory");
}
__device__ __forceinline__ bool next_cta(const void* answer, uint32_t& cta) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 a;\n\t"
        "ld.shared.b128 a, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n\t}"
        : "=r"(ok), "=r"(cta)
        : "r"(smem_u32(answer))
        : "memory");
    return ok != 0;
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
// The row's last vector, which V cuts: nothing past the row is touched.
template <int DT>
__device__ __forceinline__ uint4 load_cut(const char* row, int64_t V, int v) {
    return load_vec<DT>(row, V, v);
}

// ---- rows -----------------------------------------------------------------------

// A row as the fetching warp hands it over.
enum : int { kEnd = 0, kSkip = 1, kNone = 2, kRow = 3 };  // no more rows; not touched; without a loss; read
struct Item {
    int64_t q, o;     // its place in the logits, and in the per-row arrays
    int kind, token;
    float weight;
    float m, inv, away, k;  // gradient from the state
};

struct Shared {
    Part part[kSlots][8 * kWarps];  // every warp's of every CTA of the cluster
    Item item[kItems];
    float4 row[2];                  // maximum, 1 / sum, 1 - q of the token, slope
    uint64_t item_full[kItems], item_empty[kItems];
    uint64_t full[kMaxRing], empty[kMaxRing];
    uint64_t shares[kSlots], row_ready[2];
    uint64_t next, next_free;       // the answer to ask_next is there; every CTA has read it (in the first CTA)
    __align__(16) unsigned char answer[16];
};
__host__ __device__ inline size_t ring_offset() { return (sizeof(Shared) + 127) & ~(size_t)127; }

// Position in the ring of chunks, and the parity of its full barrier.
struct Cursor {
    int at = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void step(int n) {
        if (++at == n) {
            at = 0;
            parity ^= 1u;
        }
    }
};

template <int DT>
struct TokenSlice {
    int v0, n;        // vectors of this CTA
    int whole;        // those that V does not cut
    int chunks;
    __device__ TokenSlice(int64_t V, int split, int rank) {
        constexpr int EPV = Row<DT>::EPV;
        const int nv = (int)((V + EPV - 1) / EPV);
        const int per = ((nv + split - 1) / split + 7) & ~7;
        v0 = min(nv, rank * per);
        n = min(nv, v0 + per) - v0;
        whole = max(0, min((int)(V / EPV), v0 + n) - v0);
        chunks = (whole + kChunkVecs - 1) / kChunkVecs;
    }
};

// Running sum of a thread.
struct Running {
    float ref = -FLT_MAX;  // of the weights
    float top = -INFINITY; // the largest logit so far
    f2 sum = pack2(0.f, 0.f);
};
template <int DT, int N>
__device__ __forceinline__ void add_vectors(Running& a, const uint4 (&w)[N], f2 c2, f2 lo2, float c) {
    constexpr int EPV = Row<DT>::EPV;
    float m = Row<DT>::vmax(w[0]);
#pragma unroll
    for (int u = 1; u < N; ++u) m = max_nan(m, Row<DT>::vmax(w[u]));
    a.top = max_nan(a.top, m);
    if ((m - a.ref) * c > kRebase) {
        const float e = ex2((a.ref - m) * c);
        a.sum = mul2(a.sum, pack2(e, e));
        a.ref = m;
    }
    const f2 r2 = pack2(a.ref, a.ref);
    f2 sum[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
        float z[EPV];
        Row<DT>::unpack(w[u], z);
        f2 e[EPV / 2];
#pragma unroll
        for (int p = 0; p < EPV / 2; ++p) e[p] = weights_of(pack2(z[2 * p], z[2 * p + 1]), r2, c2, lo2);
#pragma unroll
        for (int h = EPV / 4; h; h >>= 1)
#pragma unroll
            for (int p = 0; p < h; ++p) e[p] = add2(e[p], e[p + h]);
        sum[u] = e[0];
    }
#pragma unroll
    for (int h = N / 2; h; h >>= 1)
#pragma unroll
        for (int u = 0; u < h; ++u) sum[u] = add2(sum[u], sum[u + h]);
    a.sum = add2(a.sum, sum[0]);
}

// What a row's loss is, by the warp that has its sums (lane 0 writes): its slope.
struct RowInputs {
    float weight, advantage, old_logp, ref_logp;
};
__device__ __forceinline__ RowInputs row_inputs(const TokenArgs& a, int64_t o, float weight) {
    return RowInputs{weight, a.op == kTokenPolicy ? a.advantages[o] : 0.f, a.old_logp ? a.old_logp[o] : 0.f,
                     a.ref_logp ? a.ref_logp[o] : 0.f};
}
__device__ float finish_row(const TokenArgs& a, int64_t o, const TokenRow& t, const RowInputs& in, bool write) {
    LossSlope x{0.f, in.weight};
    double term = 0.0;
    if (a.op == kTokenPolicy)
        x = policy_row(a.policy, t.logp, in.weight, in.advantage, a.old_logp != nullptr, in.old_logp, in.ref_logp);
    else if (a.op == kTokenPreference)
        term = (double)in.weight * (t.logp - (double)in.ref_logp);
    if (!write) return x.slope;
    if (!t.ok || x.slope != x.slope) raise_status(a.dev_status, DLM_DEV_NONFINITE);
    if (a.op == kTokenPolicy) a.loss[o] = x.loss;
    if (a.logp) a.logp[o] = (float)t.logp;
    if (a.lse) a.lse[o] = (float)t.lse;
    if (a.state) {
        float4* s = reinterpret_cast<float4*>(a.state + o * DLM_TOKEN_STATE);
        s[0] = make_float4(t.m, t.inv, t.away, a.op == kTokenPreference ? 0.f : x.slope);  // (a row in no pair: 0)
        s[1] = make_float4(__int_as_float(__double2loint(term)), __int_as_float(__double2hiint(term)), __int_as_float(-1), 0.f);
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

// A row's shares of all CTAs of the cluster, in slot s, and what follows from them.
__device__ __forceinline__ TokenRow merge_row(const TokenArgs& a, const Shared& sh, int s, int n) {
    const int lane = threadIdx.x & 31;
    const float c = a.scale;
    Part p = lane < n ? sh.part[s][lane] : Part{-INFINITY, 0.f, -INFINITY, 0.f};
    if (lane + 32 < n) {
        const Part b = sh.part[s][lane + 32];
        const float ref = max_nan(p.ref, b.ref), to = or_zero(ref);
        p.sum = p.sum * ex2((p.ref - to) * c) + b.sum * ex2((b.ref - to) * c);
        p.ref = ref;
        p.z = max_nan(p.z, b.z);
    }
    p = warp_part(p, c);
    return token_row(p.ref, p.sum, p.z, a.scale, a.scale_lo, a.inv_t);
}

// The fetching warp's thread: rows in the order in which the hardware gives them, their
// settings, and their slices chunk by chunk into the ring.  What the next row needs is
// asked for while this row's chunks are on their way: the row itself (about 1 us), then
// its token and weight (another), which are not looked at before the row's turn.
template <int DT, bool SUMS, bool GRAD>
struct Fetcher {
    const TokenArgs& a;
    Shared& sh;
    unsigned char* ring;
    const int rank;
    const TokenSlice<DT> sl;
    Cursor cur;
    uint32_t issued = 0;
    Item next_item{};
    uint32_t asked = 0, answers = 0;     // (asked: the first CTA's)
    bool have_next = false;                      // next_item is being read

    __device__ Fetcher(const TokenArgs& args, Shared& s, unsigned char* r, int k)
        : a(args), sh(s), ring(r), rank(k), sl(args.vocab, args.split, k) {}

    // Starts to read what belongs to row r.
    __device__ __forceinline__ void read_row(int64_t r) {
        Item& it = next_item;
        it.kind = kRow;
        it.q = r;
        if (SUMS && a.row_index) {
            it.q = a.row_index[r];
            if (it.q < 0 || (a.n_src > 0 && it.q >= a.n_src)) {
                it.kind = kSkip;
                if (rank == 0) raise_status(a.dev_status, DLM_DEV_BAD_INDEX);
            }
        }
        it.o = a.gather ? r : it.q;
        if (it.kind != kRow) return;
        it.token = a.tokens[it.o];
        if (SUMS) {
            it.weight = a.weights ? a.weights[it.o] : 1.f;
        } else {
            const float4 s = *reinterpret_cast<const float4*>(a.state + r * DLM_TOKEN_STATE);
            it.m = s.x;
            it.inv = s.y;
            it.away = s.z;
            it.k = s.w;
            it.weight = 1.f;
            if (a.grad_loss) {
                const int64_t at = a.op == kTokenPreference ? (int64_t)__float_as_int(a.state[r * DLM_TOKEN_STATE + 6]) : r;
                it.weight = at >= 0 && at < a.n_up ? a.grad_loss[at] : 0.f;
            }
        }
    }
    // The item that read_row() began.
    __device__ __forceinline__ Item row_read() {
        Item it = next_item;
        if (it.kind == kRow) {
            bool none = it.token < 0 || it.token >= a.vocab;
            if (SUMS) {
                none = none || it.weight == 0.f;
                if (it.token >= a.vocab && rank == 0) raise_status(a.dev_status, DLM_DEV_BAD_INDEX);
            } else {
                it.k *= (float)a.inv_t * it.weight;
                none = none || it.k == 0.f || it.inv == 0.f;
            }
            if (none) it.kind = kNone;
        }
        return it;
    }
    // The first CTA asks for a row once every CTA has read the last answer.
    __device__ __forceinline__ bool ask(bool block) {
        if (rank != 0 || asked > answers) return true;
        if (asked > 0) {
            const uint32_t parity = (asked - 1) & 1u;
            if (block ? !wait_for(&sh.next_free, parity) : !mbar_test_wait(&sh.next_free, parity)) return !block;
        }
        ask_next(sh.answer, &sh.next, a.split > 1);
        ++asked;
        return true;
    }
    // Takes the answer if it is there (block: waits for it).
    __device__ __forceinline__ bool look_ahead(bool block) {
        if (have_next) return ask(false);
        if (!ask(block)) return false;
        if (block ? !wait_for(&sh.next, answers & 1u) : !mbar_test_wait(&sh.next, answers & 1u)) return !block;
        uint32_t cta;
        const bool more = next_cta(sh.answer, cta);
        ++answers;
        have_next = true;
        next_item.kind = kEnd;
        if (!more) {
            asked = answers + 1;  // and nothing is asked for any more
            return true;
        }
        mbar_expect_tx(&sh.next, 16);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the answer has been read before the next one is written
        arrive_at(&sh.next_free, 0);
        read_row(cta / a.split);
        return ask(false);
    }
    __device__ bool run() {
        const int passes = SUMS && GRAD && !a.resident ? 2 : 1;
        read_row(blockIdx.x / a.split);
        for (uint32_t i = 0;; ++i) {
            const Item it = row_read();
            have_next = false;
            const int slot = i % kItems;
            if (!wait_for(&sh.item_empty[slot], ((i / kItems) & 1u) ^ 1u)) return false;
            sh.item[slot] = it;
            arrive(&sh.item_full[slot]);
            if (it.kind == kEnd) return true;
            if (it.kind == kRow) {
                const char* src = static_cast<const char*>(a.logits) + it.q * a.row_stride * Row<DT>::ESZ + (int64_t)sl.v0 * 16;
                for (int pass = 0; pass < passes; ++pass)
                    for (int c = 0; c < sl.chunks; ++c) {
                        if (!wait_for(&sh.empty[cur.at], cur.parity ^ 1u)) return false;
                        const uint32_t bytes = (uint32_t)min(kChunkVecs, sl.whole - c * kChunkVecs) * 16;
                        mbar_expect_tx(&sh.full[cur.at], bytes);
                        fetch(ring + cur.at * kChunkBytes, src + (int64_t)c * kChunkBytes, bytes, &sh.full[cur.at]);
                        cur.step(a.ring);
                        ++issued;
                        look_ahead(false);
                    }
            }
            if (!have_next && !look_ahead(true)) return false;
        }
    }
    // Copies still in flight land before the CTA ends.
    __device__ void drain() {
        Cursor c;
        for (uint32_t i = 0; i < issued; ++i) {
            if (i + a.ring >= issued) wait_for(&sh.full[c.at], c.parity);
            c.step(a.ring);
        }
        wait_for(&sh.next, answers & 1u);
    }
};

// Zeros where a row has no gradient.
template <int DT>
__device__ void write_zeros(char* out, int64_t V, const TokenSlice<DT>& sl) {
    const int t = threadIdx.x;
    uint4* dst = reinterpret_cast<uint4*>(out) + sl.v0;
    for (int v = t; v < sl.whole; v += kThreads) st_row(dst + v, make_uint4(0, 0, 0, 0));
    if (sl.whole < sl.n)
        for (int64_t e = (int64_t)(sl.v0 + sl.whole) * Row<DT>::EPV + t; e < V; e += kThreads) store_elem<DT>(out, e, 0.f);
}

// A warp of its own finishes the rows: it waits for all CTAs' shares, merges them and
// works the loss out, while the others go on.  (One of them doing this too was what a
// row took: about 2 us for each.)  With a gradient every CTA's does, to go on with the
// slope; the first CTA's writes.
template <int DT, bool GRAD>
__device__ bool finish_rows(const TokenArgs& a, Shared& sh, int rank) {
    const int lane = threadIdx.x & 31, n_parts = a.split * kWarps;
    uint32_t rows = 0;
    for (uint32_t i = 0;; ++i) {
        const int slot = i % kItems;
        if (!wait_warp(&sh.item_full[slot], (i / kItems) & 1u)) return false;
        const int kind = sh.item[slot].kind;
        const int64_t o = sh.item[slot].o;
        if (kind == kEnd) return true;
        if (kind == kNone && rank == 0 && lane == 0) finish_none(a, o);
        if (kind == kRow) {
            if (GRAD || rank == 0) {
                const RowInputs in = row_inputs(a, o, sh.item[slot].weight);
                const int ps = rows % kSlots;
                if (lane == 0) mbar_expect_tx(&sh.shares[ps], n_parts * (uint32_t)sizeof(Part));
                if (!wait_warp(&sh.shares[ps], (rows / kSlots) & 1u)) return false;
                const TokenRow x = merge_row(a, sh, ps, n_parts);
                const float slope = finish_row(a, o, x, in, rank == 0 && lane == 0);
                if (GRAD && lane == 0) {
                    sh.row[rows & 1] = make_float4(x.m, x.inv, x.away, slope);
                    arrive(&sh.row_ready[rows & 1]);
                }
            }
            ++rows;
        }
        __syncwarp();
        if (lane == 0) arrive(&sh.item_empty[slot]);
    }
}

// The arithmetic's warps: sums of their slice, the gradient.
template <int DT, bool SUMS, bool GRAD>
__device__ bool work_rows(const TokenArgs& a, Shared& sh, unsigned char* ring, int rank) {
    constexpr int EPV = Row<DT>::EPV;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int64_t V = a.vocab;
    const TokenSlice<DT> sl(V, a.split, rank);
    const float c = a.scale;
    const f2 c2 = pack2(c, c), lo2 = pack2(a.scale_lo, a.scale_lo);
    Cursor cur;
    uint32_t rows = 0;                // rows whose sums were taken so far
    for (uint32_t i = 0;; ++i) {
        const int slot = i % kItems;
        if (!wait_warp(&sh.item_full[slot], (i / kItems) & 1u)) return false;
        const Item it = sh.item[slot];
        if (it.kind == kEnd) break;
        char* out = GRAD ? static_cast<char*>(a.grad) + it.q * a.grad_stride * Row<DT>::ESZ : nullptr;
        if (it.kind == kNone) {
            if (GRAD) write_zeros<DT>(out, V, sl);
        }
        if (it.kind == kRow) {
            const char* row = static_cast<const char*>(a.logits) + it.q * a.row_stride * Row<DT>::ESZ;
            const int tv = it.token / EPV - sl.v0;        // the token's vector in the slice
            const bool mine = tv >= 0 && tv < sl.n && (tv & (kThreads - 1)) == t;
            float m = it.m, inv = it.inv, away = it.away, k = it.k;
            Cursor from = cur;
            if (SUMS) {
                Running s;
                float z_token = -INFINITY;
                for (int ch = 0; ch < sl.chunks; ++ch) {
                    if (!wait_warp(&sh.full[cur.at], cur.parity)) return false;
                    uint4* data = reinterpret_cast<uint4*>(ring + cur.at * kChunkBytes);
                    const int base = ch * kChunkVecs, n = min(kChunkVecs, sl.whole - base);
                    if (mine && tv >= base && tv < base + n) {  // the token leaves the slice (its vector is this thread's)
                        z_token = Row<DT>::scalar(data + (tv - base), it.token % EPV);
                        data[tv - base] = with_elem<DT>(data[tv - base], it.token % EPV, neg_inf_bits<DT>());
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before a copy writes here again
                    }
                    if (n == kChunkVecs) {
                        uint4 w[kPerThread];
#pragma unroll
                        for (int u = 0; u < kPerThread; ++u) w[u] = data[t + u * kThreads];
                        add_vectors<DT>(s, w, c2, lo2, c);
                    } else {
                        for (int v = t; v < n; v += kThreads) {
                            const uint4 w[1] = {data[v]};
                            add_vectors<DT>(s, w, c2, lo2, c);
                        }
                    }
                    if (!(GRAD && a.resident)) {
                        __syncwarp();
                        if (lane == 0) arrive(&sh.empty[cur.at]);
                    }
                    cur.step(a.ring);
                }
                if (sl.whole < sl.n && (sl.whole & (kThreads - 1)) == t) {  // the row's last, cut vector
                    uint4 w[1] = {load_cut<DT>(row, V, sl.v0 + sl.whole)};
                    if (mine && tv == sl.whole) {
                        z_token = Row<DT>::scalar(row, it.token);
                        w[0] = with_elem<DT>(w[0], it.token % EPV, neg_inf_bits<DT>());
                    }
                    add_vectors<DT>(s, w, c2, lo2, c);
                }
                const Part part = warp_part(Part{s.top, hsum2(s.sum) * ex2((s.ref - or_zero(s.top)) * c), z_token, 0.f}, c);
                const int ps = rows % kSlots;
                const int to = GRAD ? a.split : 1;  // every CTA, or the first
                if (lane < to) send(&sh.part[ps][rank * kWarps + warp], &sh.shares[ps], lane, part);
                if (GRAD) {
                    if (!wait_warp(&sh.row_ready[rows & 1], (rows >> 1) & 1u)) return false;
                    const float4 x = sh.row[rows & 1];
                    m = x.x;
                    inv = x.y;
                    away = x.z;
                    k = x.w * (float)a.inv_t;
                }
                ++rows;
            }
            if (GRAD) {
                if (SUMS && !a.resident) from = cur;
                const Slope slope(m, c, -k * inv);
                uint4* dst = reinterpret_cast<uint4*>(out) + sl.v0;
                for (int ch = 0; ch < sl.chunks; ++ch) {
                    if (!(SUMS && a.resident) && !wait_warp(&sh.full[from.at], from.parity)) return false;
                    const uint4* data = reinterpret_cast<const uint4*>(ring + from.at * kChunkBytes);
                    const int base = ch * kChunkVecs, n = min(kChunkVecs, sl.whole - base);
                    if (n == kChunkVecs) {
#pragma unroll
                        for (int u = 0; u < kPerThread; ++u)
                            st_row(dst + base + t + u * kThreads, slope_of<DT>(data[t + u * kThreads], slope));
                    } else {
                        for (int v = t; v < n; v += kThreads) st_row(dst + base + v, slope_of<DT>(data[v], slope));
                    }
                    __syncwarp();
                    if (lane == 0) arrive(&sh.empty[from.at]);
                    from.step(a.ring);
                }
                cur = from;
                if (sl.whole < sl.n && (sl.whole & (kThreads - 1)) == t)
                    for (int64_t e = (int64_t)(sl.v0 + sl.whole) * EPV; e < V; ++e)
                        store_elem<DT>(out, e, -k * inv * ex2((Row<DT>::scalar(row, e) - m) * c));
                if (mine) store_elem<DT>(out, it.token, k * away);  // (after this thread's own vector)
            }
        }
        __syncwarp();
        if (lane == 0) arrive(&sh.item_empty[slot]);
    }
    return true;
}

template <int DT, bool SUMS, bool GRAD>
__global__ void __launch_bounds__(kBlock, 2) token_kernel(const TokenArgs a) {
    extern __shared__ __align__(128) unsigned char s_raw[];
    Shared& sh = *reinterpret_cast<Shared*>(s_raw);
    unsigned char* ring = s_raw + ring_offset();
    const int t = threadIdx.x, rank = (int)(blockIdx.x % a.split);
    if (t == 0) {
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&sh.item_full[i], 1);
            mbar_init(&sh.item_empty[i], kWarps + (SUMS ? 1 : 0));
        }
        for (int i = 0; i < a.ring; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], kWarps);
        }
        for (int i = 0; i < kSlots; ++i) mbar_init(&sh.shares[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&sh.row_ready[i], 1);
        mbar_init(&sh.next, 1);
        mbar_init(&sh.next_free, a.split);
        mbar_init_fence();
        mbar_expect_tx(&sh.next, 16);
    }
    __syncthreads();
    if (a.split > 1) cg::this_cluster().sync();
    bool ok = true;
    if (t < kThreads) {
        ok = work_rows<DT, SUMS, GRAD>(a, sh, ring, rank);
    } else if (t < kThreads + 32) {
        if (SUMS) ok = finish_rows<DT, GRAD>(a, sh, rank);
    } else if (t == kThreads + 32) {
        Fetcher<DT, SUMS, GRAD> f(a, sh, ring, rank);
        ok = f.ask(true) && f.run();
        if (!ok) f.drain();
    }
    if (!ok) raise_status(a.dev_status, DLM_DEV_TIMEOUT);
    __syncwarp();
    if (a.split > 1) cg::this_cluster().sync();  // no CTA ends before what others send to it has come
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

namespace {

template <typename F>
cudaError_t launch_rows(F kernel, const TokenArgs& a, cudaStream_t st) {
    const size_t smem = ring_offset() + (size_t)a.ring * kChunkBytes;
    // the same limit whatever the call's size: calls may run side by side
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.n_rows * a.split));
    cfg.blockDim = dim3(kBlock);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = a.split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

// CTAs per row, and whether a step's row stays in the ring between its sums and its
// gradient.
void token_plan(TokenArgs& a, int dtype) {
    const int64_t epv = dtype == DLM_F32 ? 4 : 8, nv = (a.vocab + epv - 1) / epv;
    auto chunks = [&](int n) { return (((nv + n - 1) / n + 7) / 8 * 8 + kChunkVecs - 1) / kChunkVecs; };
    a.ring = 12;
    int split = 1;
    a.resident = 0;
    if (a.sums && a.grad) {
        while (split < 8 && chunks(split) > 5) split *= 2;
        a.resident = chunks(split) <= a.ring;
    }
    while (split < 8 && a.n_rows * split < 2LL * a.num_sms && chunks(split) > 1) split *= 2;
    a.split = split;
}

template <int DT>
cudaError_t run_token(TokenArgs a, cudaStream_t st) {
    if (a.workspace) a.state = static_cast<float*>(a.workspace);
    if (a.op == kTokenPreference && a.sums) {  // sums, the pairs, and the gradient from the state
        TokenArgs b = a;
        b.grad = nullptr;
        token_plan(b, DT);
        cudaError_t e = a.n_rows ? launch_rows(token_kernel<DT, true, false>, b, st) : cudaSuccess;
        if (e == cudaSuccess && a.n_pairs > 0) {
            pair_kernel<<<(unsigned)a.n_pairs, kThreads, 0, st>>>(a);
            e = cudaGetLastError();
        }
        if (e != cudaSuccess || !a.grad || !a.n_rows) return e;
        a.sums = 0;
    }
    token_plan(a, DT);
    if (!a.sums) return launch_rows(token_kernel<DT, false, true>, a, st);
    if (!a.grad) return launch_rows(token_kernel<DT, true, false>, a, st);
    return launch_rows(token_kernel<DT, true, true>, a, st);
}

}  // namespace

cudaError_t launch_token(const TokenArgs& a, int dtype, cudaStream_t st) {
    switch (dtype) {
    case DLM_BF16: return run_token<DLM_BF16>(a, st);
    case DLM_F16: return run_token<DLM_F16>(a, st);
    default: return run_token<DLM_F32>(a, st);
    }
}

}  // namespace dlm
