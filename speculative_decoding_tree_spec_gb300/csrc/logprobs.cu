// logprobs.cu -- what a server reports of a row of logits: the log probabilities of given tokens,
// the entropy of the distribution and its most likely tokens.
//   x = (z - max) / T,  S = sum e^x,  log p_t = x_t - ln S,  H = ln S - (sum x e^x) / S
// One pass over the row: each lane keeps its running maximum m and, referred to it, the sums of
// w = 2^a and of a w, a = (z - m) log2(e) / T.  When m grows by d (in units of a) both are carried
// over: w' = w 2^-d, a' = a - d.  Subtracting before multiplying keeps the weight of the maximum
// exactly 1; a chunk's sums (16 or 32 weights of a lane) are fp32 and join compensated sums, so that
// ln S is accurate to the weights' own rounding, and where one token holds nearly everything it
// lacks at most what that token's lane adds beside it.
//
// The most likely tokens without a list in the loop: a row is read in contiguous chunks of 2 KB, one
// warp each, and of a chunk only its largest logit is kept (one warp reduction a chunk).  Among
// contiguous chunks, ordered by (largest logit, then lower place), the k tokens wanted lie in the first
// k: a token in a later one has k better tokens before it.  So only those k chunks are read
// again (out of the L2 cache mostly), and only their elements at or above the k-th chunk's maximum are
// ranked.
//
// One CTA per row, four per SM.  A launch of fewer rows than that puts a cluster of 2, 4 or 8 CTAs on
// each row; they leave their chunks' maxima and sums in the first CTA's shared memory, which
// finishes the row.  Rows of up to 1024 logits take one warp each, the row in registers.
#include <climits>

#include <cuda_bf16.h>

#include "common.cuh"
#include "toplist.cuh"

namespace svk {

namespace {

constexpr int kLpThreads = 256;  // at most, of a CTA of the row kernel; 1024 per SM
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpPerSm = 3;     // CTAs of that size that fit an SM
constexpr int kLpUnits = 4;      // 16-byte units per lane in a load
constexpr int kLpStages = 4;     // loads of a warp in flight
constexpr int kLpMaxK = 32;
constexpr int kLpMaxCluster = 8;
constexpr int kLpSmallV = 1024;
constexpr int kLpCand = 256;     // elements ranked by counting
constexpr size_t kLpRing = kLpStages * kLpUnits * 32 * 16;  // bytes of a warp
constexpr int kLpMaxShared = (int)(kLpWarps * kLpRing) + SPEC_MAX_VOCAB / 1024 * 4;
constexpr int kLpFineV = 32768;
constexpr int kLpCount = 512;    // chunks ranked by counting

struct LogprobJob {
  const void* base;
  int64_t pitch_bytes;
  int n_rows, R, V, G, k;
  float c;      // log2(e) / T
  float inv_t;  // 1 / T
  const int32_t* rows;
  const int32_t* tokens;
  float* out_lp;
  float* out_entropy;
  int32_t* out_top;
  float* out_top_lp;
  int32_t* out_status;
  int cluster, n_chunks;
};

// Sums of 2^a and a 2^a over some elements, referred to their maximum m (in logits).
struct Part {
  float m, s_hi, s_lo, a;
};

__device__ __forceinline__ Part part_none() {
  Part p;
  p.m = -CUDART_INF_F;
  p.s_hi = p.s_lo = p.a = 0.f;
  return p;
}

// p referred to the larger maximum M.
__device__ __forceinline__ void part_raise(Part& p, float M, float c) {
  if (p.m == -CUDART_INF_F) {
    p.s_hi = p.s_lo = p.a = 0.f;
  } else if (p.m != M) {
    const float d = (p.m - M) * c;
    const float f = ex2_approx(d);
    // a p whose weights vanish must not turn an infinite d into NaN
    p.a = f > 0.f ? f * fmaf(d, p.s_hi, p.a) : 0.f;
    p.s_hi *= f;
    p.s_lo *= f;
  }
  p.m = M;
}

__device__ __forceinline__ Part warp_join(Part p, float c) {
  const float M = warp_max(p.m);
  part_raise(p, M, c);
  FF s;
  s.hi = p.s_hi;
  s.lo = p.s_lo;
  s = warp_sum_ff(s);
  p.s_hi = s.hi;
  p.s_lo = s.lo;
  p.a = warp_sum_f(p.a);
  return p;
}

// ln S: the logarithm of the high part and the low part's share of it.
__device__ __forceinline__ float part_log(const Part& p) {
  float s, e;
  two_sum(p.s_hi, p.s_lo, s, e);
  return logf(s) + e / s;
}

__device__ __forceinline__ float part_entropy(const Part& p, float log_s) {
  return log_s - 0.693147180559945f * (p.a / p.s_hi);
}

// What a row number outside the rows gives, and a row that holds NaN or +inf or is all -inf.
__device__ __forceinline__ void write_nothing(const LogprobJob& job, int r, int t, int step, float lp,
                                              float entropy, int status) {
  for (int g = t; g < job.G; g += step) job.out_lp[(int64_t)r * job.G + g] = lp;
  for (int j = t; j < job.k; j += step) {
    job.out_top[(int64_t)r * job.k + j] = -1;
    job.out_top_lp[(int64_t)r * job.k + j] = lp;
  }
  if (t == 0) {
    if (job.out_entropy) job.out_entropy[r] = entropy;
    if (job.out_status) job.out_status[r] = status;
  }
}

__device__ __forceinline__ int row_of(const LogprobJob& job, int r) {
  const int n = job.rows ? job.rows[r] : r;
  return (unsigned)n < (unsigned)job.n_rows ? n : -1;
}

// The given tokens' log probabilities; a token outside the vocabulary has none.
template <typename T>
__device__ __forceinline__ void write_given(const LogprobJob& job, const void* row, int r, int t,
                                            int step, float M, float log_s) {
  for (int g = t; g < job.G; g += step) {
    const int tok = job.tokens[(int64_t)r * job.G + g];
    float lp = -CUDART_INF_F;
    if ((unsigned)tok < (unsigned)job.V) lp = (Elt<T>::at(row, tok) - M) * job.inv_t - log_s;
    job.out_lp[(int64_t)r * job.G + g] = lp;
  }
}

__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void cluster_put(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

// The lane's units of the row's `at`-th load (2 KB of a warp); what lies past the row is -inf.
template <typename T>
__device__ __forceinline__ void load_units(const void* row, int V, int at, int lane,
                                           uint4 (&raw)[kLpUnits]) {
  constexpr int E = Elt<T>::kPerUnit;
  constexpr uint32_t kNegInf = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
  const int u0 = at * (32 * kLpUnits);
  const int full = V / E;
  if (u0 + 32 * kLpUnits <= full) {
#pragma unroll
    for (int j = 0; j < kLpUnits; ++j)
      raw[j] = __ldg(reinterpret_cast<const uint4*>(row) + u0 + j * 32 + lane);
    return;
  }
#pragma unroll
  for (int j = 0; j < kLpUnits; ++j) {
    const int u = u0 + j * 32 + lane;
    raw[j] = make_uint4(kNegInf, kNegInf, kNegInf, kNegInf);
    if (u < full) {
      raw[j] = __ldg(reinterpret_cast<const uint4*>(row) + u);
    } else if (u * E < V) {
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if constexpr (sizeof(T) == 2) {
          const unsigned short* p = static_cast<const unsigned short*>(row);
          const int i = u * E + 2 * q;
          w[q] = (i < V ? (uint32_t)p[i] : 0xFF80u) | ((i + 1 < V ? (uint32_t)p[i + 1] : 0xFF80u) << 16);
        } else {
          const int i = u * E + q;
          w[q] = i < V ? static_cast<const uint32_t*>(row)[i] : kNegInf;
        }
      }
      raw[j] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// The same on its way to shared memory, `slot` this lane's place (units 32 places apart).  A lane
// reads back only what it copied itself, so its own wait is all it needs.
template <typename T>
__device__ __forceinline__ void copy_units(const void* row, int V, int at, int lane, uint4* slot) {
  const int u0 = at * (32 * kLpUnits);
  if (u0 + 32 * kLpUnits <= V / Elt<T>::kPerUnit) {
#pragma unroll
    for (int j = 0; j < kLpUnits; ++j)
      cp_async16(slot + j * 32, reinterpret_cast<const uint4*>(row) + u0 + j * 32 + lane);
  } else {
    uint4 raw[kLpUnits];
    load_units<T>(row, V, at, lane, raw);
#pragma unroll
    for (int j = 0; j < kLpUnits; ++j) slot[j * 32] = raw[j];
  }
}

// NaN-propagating maximum of `n` of the lane's units from j0 on (constants where it is called).
template <typename T>
__device__ __forceinline__ float units_max(const uint4 (&raw)[kLpUnits], int j0, int n) {
  if constexpr (sizeof(T) == 2) {
    uint32_t none = 0xFF80FF80u;
    __nv_bfloat162 m2 = *reinterpret_cast<const __nv_bfloat162*>(&none);
#pragma unroll
    for (int j = 0; j < kLpUnits; ++j) {
      if (j < j0 || j >= j0 + n) continue;
      const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) m2 = __hmax2_nan(m2, *reinterpret_cast<const __nv_bfloat162*>(&w[q]));
    }
    const float lo = __low2float(m2), hi = __high2float(m2);
    return (lo != lo || hi != hi) ? CUDART_NAN_F : fmaxf(lo, hi);
  } else {
    float m = -CUDART_INF_F;
#pragma unroll
    for (int j = 0; j < kLpUnits; ++j) {
      if (j < j0 || j >= j0 + n) continue;
      const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
      for (int q = 0; q < 4; ++q)
        asm("max.NaN.f32 %0, %0, %1;\n" : "+f"(m) : "f"(__uint_as_float(w[q])));
    }
    return m;
  }
}

// Sums of 2^a and a 2^a over the lane's units, a = (z - m) c.  Weights that vanish (z = -inf)
// would make the second sum NaN: kMasked bounds a from below, which leaves those weights 0.
template <typename T, bool kMasked>
__device__ __forceinline__ void units_sums(const uint4 (&raw)[kLpUnits], float m, float c, float& s,
                                           float& aw) {
  constexpr int E = Elt<T>::kPerUnit;
  const float2 nm = make_float2(-m, -m), c2 = make_float2(c, c);
  float2 s0 = make_float2(0.f, 0.f), s1 = s0, a0 = s0, a1 = s0;
#pragma unroll
  for (int j = 0; j < kLpUnits; ++j) {
    float f[E];
    Elt<T>::unpack(raw[j], f);
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      float2 a = __fmul2_rn(__fadd2_rn(make_float2(f[e], f[e + 1]), nm), c2);
      if (kMasked) a = make_float2(fmaxf(a.x, -1000.f), fmaxf(a.y, -1000.f));
      const float2 w = make_float2(ex2_approx(a.x), ex2_approx(a.y));
      if ((e >> 1) & 1) {
        s1 = __fadd2_rn(s1, w);
        a1 = __ffma2_rn(a, w, a1);
      } else {
        s0 = __fadd2_rn(s0, w);
        a0 = __ffma2_rn(a, w, a0);
      }
    }
  }
  s0 = __fadd2_rn(s0, s1);
  a0 = __fadd2_rn(a0, a1);
  s = s0.x + s0.y;
  aw = a0.x + a0.y;
}

// One key of a chunk per load of it (kSub 1) or per 512 bytes (kSub kLpUnits).
template <typename T, int kSub>
__global__ void __launch_bounds__(kLpThreads, kLpPerSm) logprob_rows_kernel(LogprobJob job) {
  constexpr int E = Elt<T>::kPerUnit;
  constexpr int kKeyUnits = kLpUnits / kSub;  // units per lane that share a key
  extern __shared__ __align__(16) uint4 s_ring[];  // [warps][kLpStages][kLpUnits][32]
  __shared__ Part s_part[kLpMaxCluster * kLpWarps];
  __shared__ uint32_t s_bad;
  __shared__ uint64_t s_list[kLpCand];  // candidates, or a list of 32 per warp
  __shared__ int s_sel[kLpMaxK], s_count;
  __shared__ uint32_t s_tau;
  __shared__ float s_m, s_log;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int C = job.cluster, W = (int)blockDim.x >> 5;
  // [n_chunks kSub, rounded up to 4] order key of each chunk's largest logit
  uint32_t* const s_key = reinterpret_cast<uint32_t*>(s_ring + W * (kLpStages * kLpUnits * 32));
  uint4* const ring = s_ring + warp * (kLpStages * kLpUnits * 32) + lane;
  const int rank = blockIdx.x % C, r = blockIdx.x / C;
  const int n = row_of(job, r);
  if (n < 0) {  // the whole cluster agrees
    if (rank == 0) write_nothing(job, r, threadIdx.x, blockDim.x, -CUDART_INF_F, 0.f, SPEC_ROW_NONE);
    return;
  }
  const void* row = static_cast<const char*>(job.base) + (int64_t)n * job.pitch_bytes;
  const int V = job.V, k = job.k;
  const float c = job.c;
  // loads of a chunk: 1024 logits
  constexpr int loads = kSub > 1 ? 1 : 1024 / (32 * kLpUnits * E);
  const int n_loads = job.n_chunks * loads;
  // this warp's loads: chunk by chunk, C W chunks apart; `ahead` is the next one to copy
  const int skip = (C * W - 1) * loads;
  auto next = [&](int& at) {
    ++at;
    if (loads == 1 || at % loads == 0) at += skip;
  };
  int at = (rank * W + warp) * loads, ahead = at;
#pragma unroll
  for (int i = 0; i < kLpStages; ++i) {
    if (ahead < n_loads) copy_units<T>(row, V, ahead, lane, ring + i * (kLpUnits * 32));
    cp_async_commit();
    next(ahead);
  }
  if (threadIdx.x == 0) {
    s_bad = 0u;
    s_count = 0;
  }
  if (C > 1) cluster_arrive();  // the first CTA is there, its words cleared
  else __syncthreads();
  bool arrived = C > 1;

  float m = -CUDART_INF_F;
  Kahan S, A;
  int bad = 0;
  uint32_t top = 0u;
  const uint32_t key0 = C > 1 ? cluster_addr(s_key, 0) : 0u;
  int stage = 0;
  while (at < n_loads) {
    uint4* const slot = ring + stage * (kLpUnits * 32);
    stage = (stage + 1) % kLpStages;
    cp_async_wait<kLpStages - 1>();
    uint4 raw[kLpUnits];
#pragma unroll
    for (int j = 0; j < kLpUnits; ++j) raw[j] = slot[j * 32];
    const int done = at;
    next(at);
    const bool last = loads == 1 || at % loads == 0;  // of its chunk
    const float um = units_max<T>(raw, 0, kLpUnits);
    bad |= (um != um);
    if (k > 0) {
      if (arrived) {
        cluster_wait();
        arrived = false;
      }
#pragma unroll
      for (int j = 0; j < kSub; ++j) {
        top = max(top, order_key(kSub == 1 ? um : units_max<T>(raw, j * kKeyUnits, kKeyUnits)));
        if (kSub > 1 || last) {
          top = __reduce_max_sync(kFull, top);
          const int i = kSub > 1 ? done * kSub + j : done / loads;
          if (lane == 0) {
            if (C > 1) cluster_put(key0 + 4u * (uint32_t)i, top);
            else s_key[i] = top;
          }
          top = 0u;
        }
      }
    }
    if (um > m) {
      if (m != -CUDART_INF_F) {
        const float d = (m - um) * c;
        const float f = ex2_approx(d);
        const float s = S.s - S.c;
        A.s = f > 0.f ? f * fmaf(d, s, A.s - A.c) : 0.f;
        A.c = 0.f;
        S.s *= f;
        S.c *= f;
      }
      m = um;
    }
    if (m != -CUDART_INF_F) {
      float s, a;
      units_sums<T, false>(raw, m, c, s, a);
      if (a != a) units_sums<T, true>(raw, m, c, s, a);
      S.add(s);
      A.add(a);
    }
    // the registers hold what the slot held
    if (ahead < n_loads) copy_units<T>(row, V, ahead, lane, slot);
    cp_async_commit();
    next(ahead);
  }
  if (arrived) cluster_wait();

  // this warp's sums to the row's first CTA
  Part p;
  p.m = m;
  const FF s = S.ff();
  p.s_hi = s.hi;
  p.s_lo = s.lo;
  p.a = A.s - A.c;
  p = warp_join(p, c);
  bad = __any_sync(kFull, bad);
  if (lane == 0) {
    const int i = rank * W + warp;
    if (C > 1) {
      const uint32_t d = cluster_addr(&s_part[i], 0);
      cluster_put(d, __float_as_uint(p.m));
      cluster_put(d + 4, __float_as_uint(p.s_hi));
      cluster_put(d + 8, __float_as_uint(p.s_lo));
      cluster_put(d + 12, __float_as_uint(p.a));
      if (bad) cluster_put(cluster_addr(&s_bad, 0), 1u);
    } else {
      s_part[i] = p;
      if (bad) s_bad = 1u;
    }
  }
  if (C > 1) {
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
  } else {
    __syncthreads();
  }

  // the k chunks with the largest maxima, in that order
  const int n_keys = job.n_chunks * kSub, kk = min(k, n_keys);
  if (kk > 0 && n_keys <= kLpCount) {
    // a chunk's place is the number of chunks before it: larger ones, and equal ones to its left
    for (int i = threadIdx.x; i < n_keys; i += blockDim.x) {
      const uint32_t mine = s_key[i];
      int before = 0;
      for (int j = 0; j < n_keys; j += 4) {
        const uint4 o = *reinterpret_cast<const uint4*>(&s_key[j]);
        // of four chunks to the left an equal one counts, of four to the right it does not
        const uint32_t than = j + 3 < i ? mine - 1u : mine;
        before += (o.x > than) + (j + 1 < n_keys && o.y > than) + (j + 2 < n_keys && o.z > than) +
                  (j + 3 < n_keys && o.w > than);
      }
      // the four around it
      for (int j = i & ~3; j < i; ++j) before += s_key[j] == mine;
      if (before < kk) {
        s_sel[before] = i;
        if (before == kk - 1) s_tau = kk == k ? mine : 0u;  // with fewer chunks than k, every element counts
      }
    }
  } else if (kk > 0 && warp == W - 1) {
    uint32_t best = 0u;
    int where = INT_MAX;
    auto look = [&]() {
      best = 0u;
      where = INT_MAX;
      for (int i = lane; i < n_keys; i += 32)
        if (s_key[i] > best) {
          best = s_key[i];
          where = i;
        }
    };
    look();
    uint32_t most = 0u;
    for (int j = 0; j < kk; ++j) {
      most = __reduce_max_sync(kFull, best);
      const int i = __reduce_min_sync(kFull, best == most ? where : INT_MAX);
      if (lane == 0) s_sel[j] = i;
      if (where == i) {
        s_key[i] = 0u;
        look();
      }
    }
    if (lane == 0) s_tau = kk == k ? most : 0u;
  }
  // the row's sums
  if (warp == 0) {
    const int parts = C * W;
    Part q = lane < parts ? s_part[lane] : part_none();
    if (lane + 32 < parts) {
      Part o = s_part[lane + 32];
      const float M = fmaxf(q.m, o.m);
      part_raise(q, M, c);
      part_raise(o, M, c);
      FF f;
      f.hi = q.s_hi;
      f.lo = q.s_lo;
      f.add(o.s_hi);
      f.add(o.s_lo);
      q.s_hi = f.hi;
      q.s_lo = f.lo;
      q.a += o.a;
    }
    q = warp_join(q, c);
    const bool finite = !s_bad && q.m != CUDART_INF_F && q.m != -CUDART_INF_F;
    if (lane == 0) {
      const float log_s = part_log(q);
      s_m = q.m;
      s_log = finite ? log_s : CUDART_NAN_F;
      if (finite) {
        if (job.out_entropy) job.out_entropy[r] = part_entropy(q, log_s);
        if (job.out_status) job.out_status[r] = SPEC_TREE_OK;
      }
    }
  }
  __syncthreads();
  const float M = s_m, log_s = s_log;
  if (log_s != log_s) {
    write_nothing(job, r, threadIdx.x, blockDim.x, CUDART_NAN_F, CUDART_NAN_F, SPEC_ROW_NONFINITE);
    return;
  }
  if (k == 0) {
    write_given<T>(job, row, r, threadIdx.x, blockDim.x, M, log_s);
    return;
  }

  // the elements at or above the k-th chunk's maximum, of the k chunks
  const uint32_t tau = s_tau;
  const int key_loads = kSub > 1 ? 1 : loads;
  const int total = kk * key_loads;
  auto look_at = [&](int i) {  // the i-th piece of the selected chunks: its load
    const int sel = s_sel[i / key_loads];
    return kSub > 1 ? sel / kSub : sel * loads + i % key_loads;
  };
  uint4 nxt[kLpUnits];
  if (warp < total) load_units<T>(row, V, look_at(warp), lane, nxt);
  write_given<T>(job, row, r, threadIdx.x, blockDim.x, M, log_s);
  for (int i = warp; i < total; i += W) {
    uint4 raw[kLpUnits];
#pragma unroll
    for (int j = 0; j < kLpUnits; ++j) raw[j] = nxt[j];
    const int l = look_at(i);
    if (i + W < total) load_units<T>(row, V, look_at(i + W), lane, nxt);
    const int only = kSub > 1 ? s_sel[i] % kSub : 0;
#pragma unroll
    for (int j = 0; j < kLpUnits; ++j) {
      if (kSub > 1 && j != only) continue;  // kSub is kLpUnits: one unit per key
      if (order_key(units_max<T>(raw, j, 1)) < tau) continue;
      float f[E];
      Elt<T>::unpack(raw[j], f);
      const int i0 = (l * (32 * kLpUnits) + j * 32 + lane) * E;
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (order_key(f[e]) >= tau && i0 + e < V) {
          const int slot = atomicAdd(&s_count, 1);
          if (slot < kLpCand)
            s_list[slot] = ((uint64_t)order_key(f[e]) << 32) | (uint64_t)(0xFFFFFFFFu - (uint32_t)(i0 + e));
        }
    }
  }
  __syncthreads();
  const int found = s_count;
  if (found <= kLpCand) {  // a candidate's place is the number of larger ones
    for (int i = threadIdx.x; i < found; i += blockDim.x) {
      const uint64_t mine = s_list[i];
      int before = 0;
      for (int j = 0; j < found; ++j) before += s_list[j] > mine;
      if (before < k) {
        const float z = key_value((uint32_t)(mine >> 32));
        job.out_top[(int64_t)r * k + before] = (int32_t)(0xFFFFFFFFu - (uint32_t)mine);
        job.out_top_lp[(int64_t)r * k + before] = (z - M) * job.inv_t - log_s;
      }
    }
    return;
  }

  // many equal ones: each warp keeps a list of its k largest
  __syncthreads();
  uint64_t L = 0ull;
  for (int i = warp; i < total; i += W) {
    const int l = look_at(i), only = kSub > 1 ? s_sel[i] % kSub : -1;
    load_units<T>(row, V, l, lane, nxt);
#pragma unroll 1
    for (int u = 0; u < kLpUnits; ++u) {
      if (only >= 0 && u != only) continue;
      const uint4 x = u == 0 ? nxt[0] : u == 1 ? nxt[1] : u == 2 ? nxt[2] : nxt[3];
      float f[E];
      Elt<T>::unpack(x, f);
      const int i0 = (l * (32 * kLpUnits) + u * 32 + lane) * E;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint32_t o = order_key(f[e]);
        const uint64_t key = ((uint64_t)o << 32) | (uint64_t)(0xFFFFFFFFu - (uint32_t)(i0 + e));
        const uint64_t lk = __shfl_sync(kFull, L, k - 1);
        const bool in = o >= tau && i0 + e < V && key > lk;
        uint32_t who = __ballot_sync(kFull, in);
        if (__popc(who) <= 6) {
          while (who) {
            const int src = __ffs(who) - 1;
            who &= who - 1;
            L = list_insert(L, __shfl_sync(kFull, key, src), k, lane);
          }
        } else {
          L = list_merge(L, warp_sort_desc(in ? key : 0ull, lane), lane);
        }
      }
    }
  }
  s_list[warp * 32 + lane] = L;
  __syncthreads();
  if (warp == 0) {
    for (int w = 1; w < W; ++w) L = list_merge(L, s_list[w * 32 + lane], lane);
    if (lane < k) {
      const float z = key_value((uint32_t)(L >> 32));
      job.out_top[(int64_t)r * k + lane] = (int32_t)(0xFFFFFFFFu - (uint32_t)L);
      job.out_top_lp[(int64_t)r * k + lane] = (z - M) * job.inv_t - log_s;
    }
  }
}

// Rows of up to 32 kE logits: a warp each, element j 32 + lane in its lane's j-th register.
template <typename T, int kE>
__global__ void __launch_bounds__(kLpThreads) logprob_small_kernel(LogprobJob job) {
  const int lane = threadIdx.x & 31;
  const int64_t r64 = (int64_t)blockIdx.x * kLpWarps + (threadIdx.x >> 5);
  if (r64 >= job.R) return;
  const int r = (int)r64;
  const int n = row_of(job, r);
  if (n < 0) {
    write_nothing(job, r, lane, 32, -CUDART_INF_F, 0.f, SPEC_ROW_NONE);
    return;
  }
  const void* row = static_cast<const char*>(job.base) + (int64_t)n * job.pitch_bytes;
  const int V = job.V, k = job.k;
  float z[kE];
  float m = -CUDART_INF_F;
  bool nan = false;
#pragma unroll
  for (int j = 0; j < kE; ++j) {
    const int i = j * 32 + lane;
    z[j] = i < V ? Elt<T>::at(row, i) : -CUDART_INF_F;
    nan |= z[j] != z[j];
    m = fmaxf(m, z[j]);
  }
  const float M = warp_max(m);
  if (__any_sync(kFull, nan) || M == CUDART_INF_F || M == -CUDART_INF_F) {
    write_nothing(job, r, lane, 32, CUDART_NAN_F, CUDART_NAN_F, SPEC_ROW_NONFINITE);
    return;
  }
  FF s;
  Part p;
  p.m = M;
  p.a = 0.f;
#pragma unroll
  for (int j = 0; j < kE; ++j) {
    const float a = fmaxf((z[j] - M) * job.c, -1000.f);
    const float w = ex2_approx(a);
    s.add(w);
    p.a = fmaf(a, w, p.a);
  }
  s = warp_sum_ff(s);
  p.s_hi = s.hi;
  p.s_lo = s.lo;
  p.a = warp_sum_f(p.a);
  const float log_s = part_log(p);
  write_given<T>(job, row, r, lane, 32, M, log_s);
  if (lane == 0) {
    if (job.out_entropy) job.out_entropy[r] = part_entropy(p, log_s);
    if (job.out_status) job.out_status[r] = SPEC_TREE_OK;
  }
  // the k largest one after another: the lane's best key, then the warp's
  uint32_t key[kE];
#pragma unroll
  for (int j = 0; j < kE; ++j) key[j] = j * 32 + lane < V ? order_key(z[j]) : 0u;
  int mine = -1;
  float mine_lp = 0.f;
  for (int t = 0; t < k; ++t) {
    uint32_t best = key[0];
    int at = lane;
#pragma unroll
    for (int j = 1; j < kE; ++j)
      if (key[j] > best) {
        best = key[j];
        at = j * 32 + lane;
      }
    const uint32_t top = __reduce_max_sync(kFull, best);
    const int i = __reduce_min_sync(kFull, best == top ? at : INT_MAX);
    if (at == i) {
#pragma unroll
      for (int j = 0; j < kE; ++j)
        if (j * 32 + lane == i) key[j] = 0u;
    }
    if (lane == t) {
      mine = i;
      mine_lp = (key_value(top) - M) * job.inv_t - log_s;
    }
  }
  if (lane < k) {
    job.out_top[(int64_t)r * k + lane] = mine;
    job.out_top_lp[(int64_t)r * k + lane] = mine_lp;
  }
}

template <typename T>
cudaError_t launch_logprobs(LogprobJob job, cudaStream_t s) {
  if (job.V <= kLpSmallV) {
    const unsigned blocks = ((unsigned)job.R + kLpWarps - 1) / kLpWarps;
    if (job.V <= 32) logprob_small_kernel<T, 1><<<blocks, kLpThreads, 0, s>>>(job);
    else if (job.V <= 256) logprob_small_kernel<T, 8><<<blocks, kLpThreads, 0, s>>>(job);
    else logprob_small_kernel<T, 32><<<blocks, kLpThreads, 0, s>>>(job);
    return cudaGetLastError();
  }
  const int per_load = 32 * kLpUnits * Elt<T>::kPerUnit;
  // a chunk is 1024 logits; a key per 512 bytes where that leaves few chunks
  const bool fine = job.V <= kLpFineV;
  const int per_chunk = fine ? per_load : 1024;
  job.n_chunks = (job.V + per_chunk - 1) / per_chunk;
  const int n_keys = job.n_chunks * (fine ? kLpUnits : 1);
  // Warps per row: a wave of rows takes as long as a warp's loads and what finishing a row costs, about 8
  // loads' time, in a cluster 12.  Measured (us, bf16 rows of 128256, k = 5): 8 rows 8.0 with 64
  // warps, 9.1 with 32, 14.5 with 8; 152 rows 13.3 with 16, 15.1 with 8, 18.7 with 32; 640 rows 40.2 with
  // 4, 41.8 with 8, 53.7 with 2; 3840 rows 188 with 8, 191 with 4, 207 with 2.
  const int64_t room = (int64_t)device_sm_count() * kLpPerSm * kLpWarps;
  const int64_t n_loads = ((int64_t)job.V + per_load - 1) / per_load;
  int W = 1, C = 1;
  int64_t least = INT64_MAX;
  for (int w = 1; w <= kLpWarps * kLpMaxCluster; w *= 2) {
    const bool cluster = w > kLpWarps;
    const int64_t waves = ((int64_t)job.R * w + room - 1) / room;
    if (w > 1 && (w > job.n_chunks || (cluster && waves > 1))) break;
    const int64_t cost = waves * ((n_loads + w - 1) / w + (cluster ? 12 : 8));
    if (cost <= least) {
      least = cost;
      W = w < kLpWarps ? w : kLpWarps;
      C = w / W;
    }
  }
  int threads = 32 * W;
  job.cluster = C;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(job.R * C));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)W * kLpRing + (job.k > 0 ? ((size_t)n_keys + 3) / 4 * 16 : 0);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = C > 1 ? 1 : 0;
  auto kernel = fine ? logprob_rows_kernel<T, kLpUnits> : logprob_rows_kernel<T, 1>;
  static bool configured[64][2] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !configured[dev][fine]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kLpMaxShared);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev][fine] = true;
  }
  return cudaLaunchKernelEx(&cfg, kernel, job);
}

}  // namespace

}  // namespace svk

using namespace svk;

extern "C" int spec_token_logprobs(const void* logits, spec_dtype dtype, int32_t n_rows, int32_t V,
                                   int64_t row_pitch, const int32_t* rows, int32_t R,
                                   const int32_t* tokens, int32_t G, int32_t k, float temperature,
                                   float* out_logprobs, float* out_entropy, int32_t* out_top_tokens,
                                   float* out_top_logprobs, int32_t* out_status,
                                   spec_stream_t stream) {
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_UNSUPPORTED_DTYPE;
  if (n_rows < 0 || R < 0 || V < 1 || G < 0 || k < 0 || k > kLpMaxK || k > V)
    return SPEC_ERR_INVALID_ARG;
  if (!rows && R > n_rows) return SPEC_ERR_INVALID_ARG;
  if (V > SPEC_MAX_VOCAB) return SPEC_ERR_TOO_LARGE;
  // log2(e) / T has to be a float
  if (!(temperature >= SPEC_LOGPROB_MIN_TEMPERATURE) || !(temperature <= 3.402823466e38f))
    return SPEC_ERR_INVALID_ARG;
  if (row_pitch < V) return SPEC_ERR_INVALID_ARG;
  if (R == 0) return SPEC_OK;
  if ((!logits && n_rows > 0) || (G > 0 && (!tokens || !out_logprobs)) ||
      (k > 0 && (!out_top_tokens || !out_top_logprobs)))
    return SPEC_ERR_INVALID_ARG;
  const int64_t es = dtype == SPEC_BF16 ? 2 : 4;
  if (row_pitch > INT64_MAX / 8) return SPEC_ERR_TOO_LARGE;
  if ((reinterpret_cast<uintptr_t>(logits) & 15u) || (row_pitch * es) % 16 != 0)
    return SPEC_ERR_MISALIGNED;
  LogprobJob job{};
  job.base = logits;
  job.pitch_bytes = row_pitch * es;
  job.n_rows = n_rows;
  job.R = R;
  job.V = V;
  job.G = G;
  job.k = k;
  job.c = (float)(1.4426950408889634 / (double)temperature);
  job.inv_t = (float)(1.0 / (double)temperature);
  job.rows = rows;
  job.tokens = tokens;
  job.out_lp = out_logprobs;
  job.out_entropy = out_entropy;
  job.out_top = out_top_tokens;
  job.out_top_lp = out_top_logprobs;
  job.out_status = out_status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      dtype == SPEC_BF16 ? launch_logprobs<uint16_t>(job, s) : launch_logprobs<float>(job, s);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
