// The router of a mixture of experts, the plan that groups its (token, choice)
// slots by expert, the weighted sum over a token's experts, SwiGLU on its own,
// and their gradients.
//
// Selection.  Expert e stands before f when its logit is larger, or equal and
// e < f.  A logit of -inf closes an expert to the token, and a NaN counts as
// one: closed experts are never chosen, so a token with fewer than k open
// experts has dropped slots (expert -1, weight 0), and a padded token, all of
// whose logits are -inf, takes part in nothing.
//
// Weights.  softmax over the open experts, p_e = exp(z_e - z_max) / sum; the
// chosen experts' p, or with `normalize` divided by their sum.
//
// Plan.  slot s = t k + j.  Row r of the grouped arrays is the r-th slot in the
// order (expert, slot): a stable counting sort, so the plan is a function of
// the logits alone.
#include "experts.h"

namespace sg {
namespace {


__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// logits as unsigned integers of the same order; 0: closed (-inf or NaN)
__device__ __forceinline__ uint32_t order_key(float z) {
    if (!(z > -__builtin_inff())) return 0;
    const uint32_t u = __float_as_uint(z + 0.0f);  // -0 + 0 = +0: equal logits have equal keys
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

// One wave, one token.  Lane l holds experts l + 64 i.  Returns the token's
// choices through `put(j, expert, weight)`, called by lane 0.
template <int V, typename Put>
__device__ __forceinline__ void choose(const Route& r, int64_t t, Put put) {
    const int lane = threadIdx.x & 63;
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 64 * i;
        key[i] = e < r.E ? order_key(load_as_f32(r.logits, r.dtype, t * r.ld + e)) : 0u;
    }
    float total = 0.f, top = 0.f;
    if (!r.normalize) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) m = max(m, key[i]);
#pragma unroll
        for (int d = 32; d; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
        top = key_value(m);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (key[i]) total += expf(key_value(key[i]) - top);
        total = wave_sum(total);
    }
    // lane j keeps choice j
    int mine = -1;
    float z = 0.f;
    for (int j = 0; j < r.k; ++j) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) m = max(m, key[i]);
#pragma unroll
        for (int d = 32; d; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
        if (m == 0) break;
        bool found = false;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (found) continue;
            const uint64_t eq = __ballot(key[i] == m);
            if (eq) {
                const int l = __builtin_ctzll(eq);
                if (lane == l) key[i] = 0;
                if (lane == j) mine = l + 64 * i, z = key_value(m);
                found = true;
            }
        }
    }
    if (r.normalize) top = __shfl(z, 0);
    float w = mine >= 0 ? expf(z - top) : 0.f;
    if (r.normalize) {
        total = 0.f;
        for (int j = 0; j < r.k; ++j) total += __shfl(w, j);
    }
    w = mine >= 0 ? w / total : 0.f;
    if (lane < r.k) put(lane, mine, w);
}

// lanes of the wave whose value equals this lane's (values below 2^bits)
__device__ __forceinline__ uint64_t same_lanes(int v, int bits) {
    uint64_t m = ~0ull;
    for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot((v >> b) & 1);
        m &= ((v >> b) & 1) ? set : ~set;
    }
    return m;
}

// ---- few slots: one workgroup does it all -----------------------------------
// Bound by latency (one launch instead of three).  16 waves choose, then the
// sort runs in LDS: each wave counts a run of slots, the counts are turned
// into first rows, and each wave places its run in slot order.
constexpr int kSmallSlots = 2048, kSmallExperts = 256;

template <int V>
__global__ __launch_bounds__(1024) void route_small_kernel(Route r) {
    __shared__ int ids[kSmallSlots];
    __shared__ int first[16][kSmallExperts];  // counts, then the first row, of a wave's run and an expert
    __shared__ int total[kSmallExperts + 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n = r.T * r.k;
    int bits = 1;
    while ((1 << bits) < r.E) ++bits;
    for (int i = tid; i < 16 * kSmallExperts; i += 1024) (&first[0][0])[i] = 0;
    for (int t = wave; t < r.T; t += 16)
        choose<V>(r, t, [&](int j, int e, float w) {
            const int s = t * r.k + j;
            ids[s] = e;
            r.experts[s] = e;
            r.weights[s] = w;
        });
    __syncthreads();
    const int run = (n + 1023) / 1024 * 64;  // slots of a wave
    const int s0 = wave * run;
    for (int i = 0; i < run; i += 64) {
        const int s = s0 + i + lane;
        const int e = s < n ? ids[s] : -1;
        const uint64_t same = same_lanes(e + 1, bits + 1);
        if (e >= 0 && lane == __builtin_ctzll(same)) first[wave][e] += __builtin_popcountll(same);
    }
    __syncthreads();
    if (tid < r.E) {
        int sum = 0;
        for (int w = 0; w < 16; ++w) {
            const int c = first[w][tid];
            first[w][tid] = sum;
            sum += c;
        }
        total[tid] = sum;
    }
    __syncthreads();
    if (wave == 0) {  // exclusive scan of the experts' totals
        int before = 0;
        for (int e0 = 0; e0 < r.E; e0 += 64) {
            const int e = e0 + lane;
            const int c = e < r.E ? total[e] : 0;
            int sum = c;
            for (int d = 1; d < 64; d *= 2) {
                const int v = __shfl_up(sum, d);
                if (lane >= d) sum += v;
            }
            if (e < r.E) {
                total[e] = before + sum - c;
                r.offsets[e] = before + sum - c;
            }
            before += __shfl(sum, 63);
        }
        if (lane == 0) {
            total[r.E] = before;
            r.offsets[r.E] = before;
        }
    }
    __syncthreads();
    for (int i = 0; i < run; i += 64) {
        const int s = s0 + i + lane;
        const int e = s < n ? ids[s] : -1;
        const uint64_t same = same_lanes(e + 1, bits + 1);
        if (e >= 0) {
            const int at = total[e] + first[wave][e] + __builtin_popcountll(same & ((1ull << lane) - 1));
            r.rows[at] = s;
            r.slots[s] = at;
        } else if (s < n) {
            r.slots[s] = -1;
        }
        // the wave's reads of `first` are done before its update (one wave, in order)
        __builtin_amdgcn_wave_barrier();
        if (e >= 0 && lane == __builtin_ctzll(same)) first[wave][e] += __builtin_popcountll(same);
        __builtin_amdgcn_wave_barrier();
    }
    for (int i = total[r.E] + tid; i < n; i += 1024) r.rows[i] = -1;
}

// ---- many slots: choose and count, scan, place ------------------------------
// Chunks of consecutive tokens; ws[chunk][expert] holds the chunk's counts,
// after the scan the chunk's first row of that expert.
template <int V>
__global__ __launch_bounds__(1024) void route_choose_kernel(Route r, int chunk_tokens) {
    __shared__ int count[kRouteMaxExperts];
    const int tid = threadIdx.x, wave = tid >> 6;
    for (int i = tid; i < r.E; i += 1024) count[i] = 0;
    __syncthreads();
    const int t0 = blockIdx.x * chunk_tokens, t1 = min(t0 + chunk_tokens, r.T);
    for (int t = t0 + wave; t < t1; t += 16)
        choose<V>(r, t, [&](int j, int e, float w) {
            const int64_t s = (int64_t)t * r.k + j;
            r.experts[s] = e;
            r.weights[s] = w;
            if (e >= 0) atomicAdd(&count[e], 1);  // counts: no order in them
        });
    __syncthreads();
    for (int i = tid; i < r.E; i += 1024) r.ws[(int64_t)blockIdx.x * r.E + i] = count[i];
}

// One workgroup: thread (part, e) walks a part of the chunks of expert e.
__global__ __launch_bounds__(1024) void route_scan_kernel(Route r, int chunks) {
    __shared__ int part_sum[1024];
    __shared__ int base[kRouteMaxExperts];
    const int tid = threadIdx.x, lane = tid & 63;
    int ep = 1;
    while (ep < r.E) ep *= 2;  // experts of a part, padded
    const int parts = 1024 / ep, e = tid % ep, part = tid / ep;
    const int per = (chunks + parts - 1) / parts;
    const int c0 = min(part * per, chunks), c1 = min(c0 + per, chunks);
    int sum = 0;
    if (e < r.E) {
#pragma unroll 8
        for (int c = c0; c < c1; ++c) sum += r.ws[(int64_t)c * r.E + e];
    }
    part_sum[tid] = sum;
    __syncthreads();
    if (tid < 64) {
        int before = 0;
        for (int e0 = 0; e0 < r.E; e0 += 64) {
            const int x = e0 + lane;
            int c = 0;
            if (x < r.E)
                for (int q = 0; q < parts; ++q) c += part_sum[q * ep + x];
            int run = c;
            for (int d = 1; d < 64; d *= 2) {
                const int v = __shfl_up(run, d);
                if (lane >= d) run += v;
            }
            if (x < r.E) {
                base[x] = before + run - c;
                r.offsets[x] = before + run - c;
            }
            before += __shfl(run, 63);
        }
        if (lane == 0) r.offsets[r.E] = before;
    }
    __syncthreads();
    if (e < r.E) {
        int at = base[e];
        for (int q = 0; q < part; ++q) at += part_sum[q * ep + e];
#pragma unroll 8
        for (int c = c0; c < c1; ++c) {
            const int64_t i = (int64_t)c * r.E + e;
            const int n = r.ws[i];
            r.ws[i] = at;
            at += n;
        }
    }
}

// One wave a chunk: 64 slots at a time, in slot order.
__global__ __launch_bounds__(64) void route_place_kernel(Route r, int chunk_tokens) {
    __shared__ int next[kRouteMaxExperts];
    const int lane = threadIdx.x;
    for (int i = lane; i < r.E; i += 64) next[i] = r.ws[(int64_t)blockIdx.x * r.E + i];
    __syncthreads();
    int bits = 1;
    while ((1 << bits) < r.E) ++bits;
    const int64_t s0 = (int64_t)blockIdx.x * chunk_tokens * r.k, n = (int64_t)r.T * r.k;
    const int64_t s1 = min(s0 + (int64_t)chunk_tokens * r.k, n);
    const int32_t total = r.offsets[r.E];
    for (int64_t b = s0; b < s1; b += 64) {
        const int64_t s = b + lane;
        const int e = s < s1 ? r.experts[s] : -1;
        const uint64_t same = same_lanes(e + 1, bits + 1);
        if (e >= 0) {
            const int at = next[e] + __builtin_popcountll(same & ((1ull << lane) - 1));
            r.rows[at] = (int32_t)s;
            r.slots[s] = at;
        } else if (s < s1) {
            r.slots[s] = -1;
        }
        __builtin_amdgcn_wave_barrier();
        if (e >= 0 && lane == __builtin_ctzll(same)) next[e] += __builtin_popcountll(same);
        __builtin_amdgcn_wave_barrier();
        if (s < s1 && s >= total) r.rows[s] = -1;
    }
}

// ---- gradient of the router -------------------------------------------------
// With g_e the gradient of the weight of expert e (0 where not chosen) and q
// the distribution the weights come from (the chosen experts' own with
// `normalize`, else the softmax over the open experts):
//   dz_e = q_e (g_e - sum_f q_f g_f)
// One wave a token; the sum over the chosen experts in choice order.
template <int V>
__global__ __launch_bounds__(256) void route_backward_kernel(Route r, const float* dweights, void* dlogits,
                                                             int64_t ldd) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= r.T) return;
    int ej = -1;
    float wj = 0.f, dj = 0.f;
    if (lane < r.k) {
        ej = r.experts[t * r.k + lane];
        if (ej >= 0 && ej < r.E) wj = r.weights[t * r.k + lane], dj = dweights[t * r.k + lane];
        else ej = -1;
    }
    const float prod = ej >= 0 ? wj * dj : 0.f;
    float back = 0.f;
    for (int j = 0; j < r.k; ++j) back += __shfl(prod, j);
    uint32_t key[V];
    float p[V];
    if (!r.normalize) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 64 * i;
            key[i] = e < r.E ? order_key(load_as_f32(r.logits, r.dtype, t * r.ld + e)) : 0u;
            m = max(m, key[i]);
        }
#pragma unroll
        for (int d = 32; d; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
        const float top = key_value(m);
        float total = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] = key[i] ? expf(key_value(key[i]) - top) : 0.f;
            total += p[i];
        }
        total = wave_sum(total);
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = key[i] ? -(p[i] / total) * back : 0.f;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = 0.f;
    }
    for (int j = 0; j < r.k; ++j) {
        const int e = __shfl(ej, j);
        const float w = __shfl(wj, j), d = __shfl(dj, j);
        if (e < 0) continue;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (e == lane + 64 * i) p[i] = w * (d - back);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 64 * i;
        if (e < r.E) store_from_f32(dlogits, r.dtype, t * ldd + e, p[i]);
    }
}

// ---- weighted sum of a token's rows ----------------------------------------
// out[t] = sum_j w[t][j] y[slots[t][j]] in choice order, dropped slots left
// out.  Bound by HBM: every row read once, every output written once.  A
// thread owns 8 adjacent columns.
// WHOLE: D is a multiple of 8 (with a branch for the row's end between them the
// loads do not go out together: the gradient below 104 -> 161 us).
template <int YT, int OT, bool WHOLE>
__global__ __launch_bounds__(256) void combine_kernel(const void* y, const int32_t* slots, const float* weights, int k,
                                                      int64_t D, int64_t R, void* out, int per_token) {
    const int64_t t = blockIdx.x / per_token;
    const int64_t c = ((int64_t)(blockIdx.x - t * per_token) * blockDim.x + threadIdx.x) * 8;
    if (c >= D) return;
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int j0 = 0; j0 < k; j0 += 4) {  // four rows' loads at once
        float v[4][8], w[4];
        bool in[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t s = t * k + min(j0 + j, k - 1), row = slots[s];
            in[j] = j0 + j < k && row >= 0 && row < R;
            w[j] = weights ? weights[s] : 1.f;
            if (in[j]) load_cols<YT>(y, row * D + c, v[j], WHOLE ? 8 : D - c);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (in[j])
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = fmaf(w[j], v[j][e], acc[e]);
    }
    store_cols<OT>(out, t * D + c, acc, WHOLE ? 8 : (int)min(D - c, (int64_t)8));
}

// ---- its gradient -----------------------------------------------------------
// dy[slots[t][j]] = w[t][j] dout[t], dw[t][j] = <dout[t], y[slots[t][j]]>.
// One workgroup a token: its dout is read once per choice from the caches, the
// rows of y once.  The dot products are summed over lanes in a fixed tree.
template <int DT, bool WHOLE>
__global__ __launch_bounds__(256) void combine_backward_kernel(const void* dout, const void* y,
                                                               const int32_t* __restrict__ slots,
                                                               const float* __restrict__ weights, int k, int64_t D, int64_t R,
                                                               void* dy, float* dw) {
    __shared__ float part[kRouteMaxK][4];
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // (lane j holds slot j: no load of it waits behind the rows')
    const int mine = lane < k ? slots[t * k + lane] : -1;
    const float wmine = lane < k && weights ? weights[t * k + lane] : 1.f;
    for (int j = 0; j < k; ++j) {
        const int64_t row = __builtin_amdgcn_readlane(mine, j);
        const bool ok = row >= 0 && row < R;
        float dot = 0.f;
        if (ok) {
            const float w = __shfl(wmine, j);
            for (int64_t c = (int64_t)threadIdx.x * 8; c < D; c += 256 * 8) {
                float g[8], v[8], o[8];
                load_cols<DT>(dout, t * D + c, g, WHOLE ? 8 : D - c);
                if (dw) {
                    load_cols<DT>(y, row * D + c, v, WHOLE ? 8 : D - c);
#pragma unroll
                    for (int e = 0; e < 8; ++e) dot = fmaf(g[e], v[e], dot);
                }
                if (dy) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = w * g[e];
                    store_cols<DT>(dy, row * D + c, o, WHOLE ? 8 : (int)min(D - c, (int64_t)8));
                }
            }
        }
        if (dw) {
            dot = wave_sum(dot);
            if (lane == 0) part[j][wave] = dot;
        }
    }
    if (dw) {
        __syncthreads();
        if (threadIdx.x < (unsigned)k)
            dw[t * k + threadIdx.x] = (part[threadIdx.x][0] + part[threadIdx.x][1]) +
                                      (part[threadIdx.x][2] + part[threadIdx.x][3]);
    }
}

// ---- SwiGLU on stored gate | up rows ---------------------------------------
// h = silu(g) u;  with s = 1 / (1 + e^-g): dg = dh u s (1 + g (1 - s)),
// du = dh g s.  Bound by HBM.
template <int DT, bool BWD, bool WHOLE>
__global__ __launch_bounds__(256) void swiglu_kernel(const void* gu, const void* dh, int64_t rows, int64_t f,
                                                     int64_t fc, void* out) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= rows * fc) return;
    const int64_t row = i / fc, c = (i - row * fc) * 8;
    const int left = WHOLE ? 8 : (int)min(f - c, (int64_t)8);
    float g[8], u[8], a[8], b[8];
    auto part = [&](int64_t base, float(&v)[8], const void* p) { load_cols<DT>(p, base + c, v, left); };
    auto put = [&](int64_t base, const float(&v)[8]) { store_cols<DT>(out, base + c, v, left); };
    part(row * 2 * f, g, gu);
    part(row * 2 * f + f, u, gu);
    if constexpr (!BWD) {
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] = silu_f32(g[e]) * u[e];
        put(row * f, a);
    } else {
        float d[8];
        part(row * f, d, dh);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float s = 1.0f / (1.0f + expf(-g[e]));
            a[e] = d[e] * u[e] * s * (1.0f + g[e] * (1.0f - s));
            b[e] = d[e] * g[e] * s;
        }
        put(row * 2 * f, a);
        put(row * 2 * f + f, b);
    }
}

bool small(int64_t T, int E, int k) { return T * k <= kSmallSlots && T <= 256 && E <= kSmallExperts; }

int chunk_tokens_of(int64_t T, int k) {
    // about 256 slots a chunk, at most 1024 chunks
    int64_t c = (256 + k - 1) / k;
    const int64_t least = (T + 1023) / 1024;
    return (int)(c > least ? c : least);
}

template <int V>
void route_v(const Route& r, hipStream_t s) {
    if (small(r.T, r.E, r.k)) {
        launch(route_small_kernel<V>, dim3(1), dim3(1024), 0, s, r);
        return;
    }
    const int ct = chunk_tokens_of(r.T, r.k);
    const int chunks = (r.T + ct - 1) / ct;  // (0 without tokens: the scan alone, which writes the offsets)
    if (chunks) launch(route_choose_kernel<V>, dim3(chunks), dim3(1024), 0, s, r, ct);
    launch(route_scan_kernel, dim3(1), dim3(1024), 0, s, r, chunks);
    if (chunks) launch(route_place_kernel, dim3(chunks), dim3(64), 0, s, r, ct);
}

}  // namespace

size_t route_workspace_ints(int64_t T, int E, int k) {
    if (small(T, E, k)) return 0;
    const int64_t ct = chunk_tokens_of(T, k);
    return (size_t)((T + ct - 1) / ct) * E;
}

hipError_t launch_route(const Route& r, hipStream_t s) {
    if (r.E <= 64) route_v<1>(r, s);
    else if (r.E <= 128) route_v<2>(r, s);
    else if (r.E <= 256) route_v<4>(r, s);
    else if (r.E <= 512) route_v<8>(r, s);
    else route_v<16>(r, s);
    return hipGetLastError();
}

hipError_t launch_route_backward(const Route& r, const float* dweights, void* dlogits, int64_t ldd, hipStream_t s) {
    const dim3 grid((unsigned)((r.T + 3) / 4));
    if (r.E <= 64) launch(route_backward_kernel<1>, grid, dim3(256), 0, s, r, dweights, dlogits, ldd);
    else if (r.E <= 128) launch(route_backward_kernel<2>, grid, dim3(256), 0, s, r, dweights, dlogits, ldd);
    else if (r.E <= 256) launch(route_backward_kernel<4>, grid, dim3(256), 0, s, r, dweights, dlogits, ldd);
    else if (r.E <= 512) launch(route_backward_kernel<8>, grid, dim3(256), 0, s, r, dweights, dlogits, ldd);
    else launch(route_backward_kernel<16>, grid, dim3(256), 0, s, r, dweights, dlogits, ldd);
    return hipGetLastError();
}

hipError_t launch_combine(const void* y, int y_dtype, const int32_t* slots, const float* weights, int64_t T, int k,
                          int64_t D, int64_t R, void* out, int out_dtype, hipStream_t s) {
    const int threads = D >= 2048 ? 256 : D >= 1024 ? 128 : 64;
    const int per = (int)((D + threads * 8 - 1) / (threads * 8));
    const dim3 grid((unsigned)(T * per));
    auto go = [&](auto yt, auto ot) {
        constexpr int YT = decltype(yt)::value, OT = decltype(ot)::value;
        if (D % 8 == 0) launch(combine_kernel<YT, OT, true>, grid, dim3(threads), 0, s, y, slots, weights, k, D, R, out, per);
        else launch(combine_kernel<YT, OT, false>, grid, dim3(threads), 0, s, y, slots, weights, k, D, R, out, per);
    };
    auto with_out = [&](auto yt) {
        if (out_dtype == SG_F32) go(yt, std::integral_constant<int, SG_F32>{});
        else if (out_dtype == SG_BF16) go(yt, std::integral_constant<int, SG_BF16>{});
        else go(yt, std::integral_constant<int, SG_F16>{});
    };
    if (y_dtype == SG_F32) with_out(std::integral_constant<int, SG_F32>{});
    else if (y_dtype == SG_BF16) with_out(std::integral_constant<int, SG_BF16>{});
    else with_out(std::integral_constant<int, SG_F16>{});
    return hipGetLastError();
}

hipError_t launch_combine_backward(const void* dout, const void* y, int dtype, const int32_t* slots,
                                   const float* weights, int64_t T, int k, int64_t D, int64_t R, void* dy, float* dw,
                                   hipStream_t s) {
    const dim3 grid((unsigned)T);
    auto go = [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        if (D % 8 == 0) launch(combine_backward_kernel<DT, true>, grid, dim3(256), 0, s, dout, y, slots, weights, k, D, R, dy, dw);
        else launch(combine_backward_kernel<DT, false>, grid, dim3(256), 0, s, dout, y, slots, weights, k, D, R, dy, dw);
    };
    if (dtype == SG_F32) go(std::integral_constant<int, SG_F32>{});
    else if (dtype == SG_BF16) go(std::integral_constant<int, SG_BF16>{});
    else go(std::integral_constant<int, SG_F16>{});
    return hipGetLastError();
}

template <bool BWD>
static hipError_t swiglu_any(const void* gu, const void* dh, int dtype, int64_t rows, int64_t f, void* out,
                             hipStream_t s) {
    const int64_t fc = (f + 7) / 8;
    const dim3 grid((unsigned)((rows * fc + 255) / 256));
    auto go = [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        if (f % 8 == 0) launch(swiglu_kernel<DT, BWD, true>, grid, dim3(256), 0, s, gu, dh, rows, f, fc, out);
        else launch(swiglu_kernel<DT, BWD, false>, grid, dim3(256), 0, s, gu, dh, rows, f, fc, out);
    };
    if (dtype == SG_F32) go(std::integral_constant<int, SG_F32>{});
    else if (dtype == SG_BF16) go(std::integral_constant<int, SG_BF16>{});
    else go(std::integral_constant<int, SG_F16>{});
    return hipGetLastError();
}
hipError_t launch_swiglu(const void* gu, int dtype, int64_t rows, int64_t f, void* h, hipStream_t s) {
    return swiglu_any<false>(gu, nullptr, dtype, rows, f, h, s);
}
hipError_t launch_swiglu_backward(const void* gu, const void* dh, int dtype, int64_t rows, int64_t f, void* dgu,
                                  hipStream_t s) {
    return swiglu_any<true>(gu, dh, dtype, rows, f, dgu, s);
}

}  // namespace sg
