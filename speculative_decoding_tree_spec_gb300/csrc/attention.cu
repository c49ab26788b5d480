// attention.cu -- attention of draft trees, single tokens and prompts over a paged cache:
// the few-rows kernel, the join of split tiles, and the entry point.
//
//   out = sum_t p_t v_t / sum_t p_t,  p_t = 2^(c q.k_t - m),  c = scale log2(e),
// in one pass over the keys with a running maximum m: when it rises the sum and the output
// taken so far are scaled by 2^(m_old - m_new).  A part of the keys gives (m, l, o); two
// parts join as m = max, l = l1 2^(m1 - m) + l2 2^(m2 - m), o likewise.
#include <cuda_bf16.h>

#include <cfloat>
#include <cmath>

#include "attention.cuh"

namespace svk {

namespace {

constexpr int kRowsR = kAttnRowsTile;  // rows of a tile: one m16 fragment
constexpr int kRowsWarps = 4;    // each takes every fourth group of keys
constexpr int kRowsThreads = 32 * kRowsWarps;
constexpr int kGroup = 16;       // keys of a warp's step
constexpr int kRowsKB = kGroup * kRowsWarps;
constexpr int kRowsC = 2;        // a tile's fixed costs in blocks
constexpr int kMaxSplit = 8;     // CTAs of a cluster that share a tile
constexpr int kSplitBlocks = 8;  // blocks of a tile that a CTA of a cluster takes at most
constexpr int kCombineThreads = 512;

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo with both parts tf32: the products hi hi + hi lo + lo hi carry an fp32
// product to about 2^-21.  The tensor cores' own sum cuts bits off where an fp32 add rounds, so
// each step of 8 starts from 0 and is added to the running sums in fp32.
//
// hi is x cut to tf32's 10 bits, lo the rest rounded to as many.  An infinite x gives hi = x and
// a finite lo (the minimum with a bound that no finite x's lo reaches drops inf - inf), and a NaN
// whose payload lies in the cut bits looks like an infinity.  The cross products with an infinite
// hi are NaN where the other operand's lo is 0, so a result that is not finite is taken again
// without the split: plain_score, take_nonfinite.
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xffffe000u;
  const float rest = fminf(x - __uint_as_float(hi), 0x1p117f);
  asm("cvt.rna.tf32.f32 %0, %1;\n" : "=r"(lo) : "f"(rest));
}

// ---------------------------------------------------------------------------------------
// Few rows (a tile of 16): what a single token's heads need, and every size or page length
// the tensor-memory kernel does not take.  Each of the four warps walks its own groups of 16
// keys with its own copies in flight, its own m, l and o, so no barrier stands in the loop;
// the four are joined at the end of the tile.  The products are warp-level matrix
// instructions: at 16 rows the keys' bytes, not the products, set the time.  fp32 inputs are
// split into two tf32 parts each.  64 requests of 1 to 8192 positions, one token each (1.07 GB):
// 197 us and 6 us for the join, 5.4 TB/s; deeper or earlier copies, cache layouts with a head's
// positions together and page numbers read further ahead change nothing in that.
//
// Two ways to cut the work.  SPLIT = false: the work list of attention.cuh, even whatever the
// lengths are, with the join in a second kernel.  SPLIT = true, for few or short tiles (see
// launch_rows): a cluster of CTAs takes one tile, each an equal run of its blocks, and joins
// the parts through distributed shared memory: no work list, no second launch.
// ---------------------------------------------------------------------------------------
template <typename T, int DP>
struct RowsCfg {
  static constexpr int kRowBytes = DP * (int)sizeof(T);
  static constexpr int kChunks = kRowBytes / 16;
  static constexpr int kStageBytes = 2 * kGroup * kRowBytes;  // keys and values
  static constexpr int kStages = 3;
  static constexpr int kQBytes = sizeof(T) == 4 ? 2 * kRowsR * DP * 4 : 0;  // split in two
  static constexpr int kSmem = kRowsWarps * kStages * kStageBytes + kQBytes;
  static constexpr int kCtasPerSm = kSmem > 110 * 1024 ? 1 : 2;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::
                   : "memory");
}
__device__ __forceinline__ float ld_cluster(const float* p, uint32_t rank) {
  uint32_t a;
  float x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(x) : "r"(a) : "memory");
  return x;
}
__device__ __forceinline__ float4 ld_cluster4(const float* p, uint32_t rank) {
  uint32_t a;
  float4 x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
               : "r"(a)
               : "memory");
  return x;
}

// Joins (ms, ls, x) to (m, l, o).
template <int C>
__device__ __forceinline__ void join_part(float& m, float& l, float (&o)[C], float ms, float ls,
                                          const float (&x)[C]) {
  if (ms == -CUDART_INF_F && ls == 0.f) return;  // sees none of these keys (NaN goes on)
  const float mn = fmaxf(m, ms);
  const float a = m == -CUDART_INF_F ? 0.f : exp2f(m - mn), b = exp2f(ms - mn);
  l = l * a + ls * b;
#pragma unroll
  for (int i = 0; i < C; ++i) o[i] = o[i] * a + x[i] * b;
  m = mn;
}

// q . k without the split, for scores that are not finite: k in shared memory, its 16-byte units
// swizzled by the key's number.
static __device__ __noinline__ float plain_score(const float* q, const unsigned char* k, int key,
                                                 int D) {
  float s = 0.f;
  for (int d = 0; d < D; ++d)
    s = fmaf(q[d], *reinterpret_cast<const float*>(k + (((d >> 2) ^ (key & 7)) << 4) + (d & 3) * 4),
             s);
  return s;
}

// The columns of o that are not finite, from the positions [from, to), which all rows of the tile
// see: where values among them are infinite or NaN, their sum is the result, whatever their
// weights are.  (Else the column is left: scores that are NaN, or an overflow.)
template <int C>
static __device__ __noinline__ void take_nonfinite(const AttnJob& job, const AttnTile& t, int head,
                                                   int from, int to, int c0, float* o) {
  const int32_t* row = job.table + (int64_t)t.b * job.max_pages;
  float sum[C];
  unsigned odd = 0, found = 0;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    sum[i] = 0.f;
    if (!(fabsf(o[i]) < CUDART_INF_F) && c0 + i < job.D) odd |= 1u << i;
  }
  for (int pos = from; pos < to; ++pos) {
    const int64_t off = paged_offset(row, job.max_pages, job.n_pages, job.pd, job.page_stride,
                                     job.pos_stride, pos);
    if (off < 0) continue;
    const float* v = static_cast<const float*>(job.v) + off + head * job.head_stride + c0;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      if (!((odd >> i) & 1u)) continue;
      const float x = v[i];
      if (!(fabsf(x) < CUDART_INF_F)) {
        sum[i] += x;
        found |= 1u << i;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < C; ++i)
    if ((found >> i) & 1u) o[i] = sum[i];
}

template <typename T, int DP, bool SPLIT>
__global__ void __launch_bounds__(kRowsThreads) attn_rows_kernel(AttnJob job) {
  using Cfg = RowsCfg<T, DP>;
  constexpr bool F32 = sizeof(T) == 4;
  constexpr int RB = Cfg::kRowBytes, CH = Cfg::kChunks, S = Cfg::kStages;
  extern __shared__ __align__(16) unsigned char attn_dyn[];
  __shared__ int poison;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gr = lane >> 2, tq = lane & 3;  // fragment row, column pair
  const int cta = blockIdx.x;
  AttnRange range{0, 0, 0, 0};
  if (!SPLIT) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may line up
    range = attn_range<kRowsR, kRowsKB, kRowsC, kRowsThreads>(job, cta, gridDim.x);
  } else {
    const int tile = cta / (int)cluster_size();
    range.units = 1;  // one walk
    range.head = tile / job.entries;
    range.entry = tile - range.head * job.entries;
  }
  if (threadIdx.x == 0) poison = 0;
  __syncthreads();
  int4 desc = make_int4(0, 0, 0, kSlotNone);
  unsigned char* ring = attn_dyn + warp * S * Cfg::kStageBytes;
  const uint32_t ring_u = smem_u32(ring);
  uint32_t* sq = reinterpret_cast<uint32_t*>(attn_dyn + kRowsWarps * S * Cfg::kStageBytes);
  const float c = job.scale_log2;

  for (AttnWalk<kRowsC> walk(range); walk.left > 0; walk.next(job)) {
    const AttnTile t = attn_tile<kRowsR, kRowsKB>(job, walk.entry);
    const int head = walk.head, entry = walk.entry;
    int block, nb;
    if (SPLIT) {
      const int rank = (int)cluster_rank(), size = (int)cluster_size();
      block = t.blocks * rank / size;
      nb = t.blocks * (rank + 1) / size - block;
      walk.left = 0;
    } else {
      walk.take(t.blocks);
      block = walk.first;
      nb = walk.blocks;
    }
    const int32_t* table_row = job.table + (int64_t)t.b * job.max_pages;
    const T* kh = static_cast<const T*>(job.k) + head * job.head_stride;
    const T* vh = static_cast<const T*>(job.v) + head * job.head_stride;
    const int seg0 = t.kbeg + block * kRowsKB;
    const int seg1 = min(seg0 + nb * kRowsKB, t.kend);

    // this thread's two rows
    int node[2];
    bool real[2];
    const T* qrow[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int b, g;
      real[i] = attn_row(job, t, t.row0 + gr + 8 * i, b, node[i], g);
      qrow[i] = static_cast<const T*>(job.q) + b * job.lq.batch_stride +
                node[i] * job.lq.node_stride + (head * job.G + g) * job.lq.head_stride;
    }
    // queries: bf16 fragments in registers, fp32 rows in shared memory
    uint32_t qa[F32 ? 1 : DP / 16][4];
    if (!F32) {
#pragma unroll
      for (int ks = 0; ks < DP / 16; ++ks)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int d = ks * 16 + 2 * tq + 8 * (i >> 1);
          qa[F32 ? 0 : ks][i] = (real[i & 1] && d < job.D)
                                    ? *reinterpret_cast<const uint32_t*>(qrow[i & 1] + d)
                                    : 0u;
        }
    } else {
      for (int i = threadIdx.x; i < kRowsR * DP; i += kRowsThreads) {
        const int r = i / DP, d = i - r * DP;
        int b, n, g;
        float x = 0.f;
        if (attn_row(job, t, t.row0 + r, b, n, g) && d < job.D)
          x = Elt<float>::at(static_cast<const float*>(job.q) + b * job.lq.batch_stride +
                                 n * job.lq.node_stride + (head * job.G + g) * job.lq.head_stride, d);
        // columns rotated by the row: the fragment reads below touch all banks
        const int at = r * DP + ((d + 4 * r) & (DP - 1));
        split_tf32(x, sq[at], sq[kRowsR * DP + at]);
      }
      __syncthreads();
    }

    // ---- this warp's groups: keys seg0 + 16 (4 i + warp) .. + 15 ----
    const int groups = nb;
    // The page of this lane's key (lane < 16) of the next group to be issued, read a group
    // ahead and not looked at before: the read's latency hides behind the group between.
    int page_next = -1, slot_next = 0;
    auto lookup = [&](int i) {
      const int pos = seg0 + (i * kRowsWarps + warp) * kGroup + lane;
      page_next = -1;
      if (i < groups && lane < kGroup && pos < seg1) {
        const int at = job.pd.div(pos);  // below max_pages: seg1 lies within the table
        page_next = table_row[at];
        slot_next = pos - at * job.pd.size;
      }
    };
    unsigned ok_ring[S];  // per stage: keys that exist
    auto issue = [&](int i, int stage) {
      const uint32_t dst = ring_u + stage * Cfg::kStageBytes;
      const bool exists = (unsigned)page_next < (unsigned)job.n_pages;
      const unsigned ok = __ballot_sync(kFull, exists);
      const int64_t off_mine = exists ? (int64_t)page_next * job.page_stride +
                                            (int64_t)slot_next * job.pos_stride
                                      : (int64_t)-1;
#pragma unroll
      for (int s = 0; s < S; ++s)
        if (s == stage) ok_ring[s] = ok;
      constexpr int rows_step = CH >= 32 ? 1 : 32 / CH;
      const int ch0 = lane % CH, r0 = lane / (CH >= 32 ? 32 : CH);
      if (i < groups) {
#pragma unroll
        for (int rr = 0; rr < kGroup; rr += rows_step) {
          const int r = rr + r0;
          const int64_t off = __shfl_sync(kFull, off_mine, r);
#pragma unroll
          for (int cc = 0; cc < CH; cc += 32) {
            const int ch = ch0 + cc;
            const bool there = off >= 0 && ch * (16 / (int)sizeof(T)) < job.D;
            const int64_t at = there ? off + ch * (16 / (int)sizeof(T)) : 0;
            const uint32_t to = dst + r * RB + ((ch ^ (r & 7)) << 4);
            cp_async16_or_zero(to, kh + at, there);
            cp_async16_or_zero(to + kGroup * RB, vh + at, there);
          }
        }
      }
      cp_async_commit();
      lookup(i + 1);
    };

    float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f};
    float o[DP / 8][4];
#pragma unroll
    for (int i = 0; i < DP / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

    lookup(0);
#pragma unroll
    for (int s = 0; s < S - 1; ++s) issue(s, s);
    int stage = 0;
    for (int i = 0; i < groups; ++i) {
      cp_async_wait<S - 2>();
      __syncwarp();
      const int pos0 = seg0 + (i * kRowsWarps + warp) * kGroup;
      unsigned ok = 0;
#pragma unroll
      for (int s = 0; s < S; ++s)
        if (s == stage) ok = ok_ring[s];
      const uint32_t sk = ring_u + stage * Cfg::kStageBytes, sv = sk + kGroup * RB;
      const unsigned char* sk_p = ring + stage * Cfg::kStageBytes;
      const unsigned char* sv_p = sk_p + kGroup * RB;
      const bool whole = ok == 0xffffu && pos0 + kGroup <= t.clear;
      if (pos0 + kGroup > t.clear) {
        // drafts among the keys: values that are not finite leave the product
        bool bad = false;
        for (int u = lane; u < kGroup * CH; u += 32) {
          if (pos0 + u / CH < t.clear) continue;
          uint4* p = reinterpret_cast<uint4*>(const_cast<unsigned char*>(sv_p)) + u;
          const uint4 x = *p;
          if (unit_nonfinite<T>(x)) {
            bad = true;
            uint32_t w[4] = {x.x, x.y, x.z, x.w};
            for (int e = 0; e < 4; ++e) {
              if (F32) {
                if ((w[e] & 0x7f800000u) == 0x7f800000u) w[e] = 0u;
              } else {
                if ((w[e] & 0x7f800000u) == 0x7f800000u) w[e] &= 0xffffu;
                if ((w[e] & 0x7f80u) == 0x7f80u) w[e] &= 0xffff0000u;
              }
            }
            *p = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        if (bad) poison = 1;
        __syncwarp();
      }

      // scores of 16 rows x 16 keys
      float s[2][4] = {};
      if (!F32) {
        // matrices: keys 0-7 / 8-15 x the two halves of a 16-wide step
        const int krow = (lane & 7) + ((lane >> 4) << 3), khalf = (lane >> 3) & 1;
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks) {
          uint32_t kb[4];
          ldmatrix_x4(kb, sk + krow * RB + (((2 * ks + khalf) ^ (krow & 7)) << 4));
          mma_bf16(s[0], qa[F32 ? 0 : ks], kb[0], kb[1]);
          mma_bf16(s[1], qa[F32 ? 0 : ks], kb[2], kb[3]);
        }
      } else {
#pragma unroll 4
        for (int ks = 0; ks < DP / 8; ++ks) {
          uint32_t ah[4], al[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = gr + 8 * (e & 1), d = ks * 8 + tq + 4 * (e >> 1);
            const int at = r * DP + ((d + 4 * r) & (DP - 1));
            ah[e] = sq[at];
            al[e] = sq[kRowsR * DP + at];
          }
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            const int key = nt * 8 + gr;
            uint32_t bh[2], bl[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float x = *reinterpret_cast<const float*>(
                  sk_p + key * RB + (((2 * ks + e) ^ (key & 7)) << 4) + tq * 4);
              split_tf32(x, bh[e], bl[e]);
            }
            float part[4] = {};
            mma_tf32(part, al, bh[0], bh[1]);
            mma_tf32(part, ah, bl[0], bl[1]);
            mma_tf32(part, ah, bh[0], bh[1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][e] += part[e];
          }
        }
        bool odd = false;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) odd |= !(fabsf(s[nt][e]) < CUDART_INF_F);
        if (odd) {
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = nt * 8 + 2 * tq + (e & 1);
              if (real[e >> 1] && !(fabsf(s[nt][e]) < CUDART_INF_F))
                s[nt][e] = plain_score(reinterpret_cast<const float*>(qrow[e >> 1]),
                                       sk_p + key * RB, key, job.D);
            }
        }
        __syncwarp();
      }
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] *= c;
      if (!whole) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = nt * 8 + 2 * tq + (e & 1), pos = pos0 + key;
            bool sees = (ok >> key) & 1u;
            if (sees && pos >= t.prefix) sees = attn_sees_draft(job, t, node[e >> 1], pos);
            if (!sees) s[nt][e] = -CUDART_INF_F;
          }
      }
      // running maximum and sum of the two rows
      float mu[2];
#pragma unroll
      for (int i2 = 0; i2 < 2; ++i2) {
        float x = fmaxf(fmaxf(s[0][2 * i2], s[0][2 * i2 + 1]), fmaxf(s[1][2 * i2], s[1][2 * i2 + 1]));
        x = fmaxf(x, __shfl_xor_sync(kFull, x, 1));
        x = fmaxf(x, __shfl_xor_sync(kFull, x, 2));
        const float mn = fmaxf(m[i2], x);
        mu[i2] = mn == -CUDART_INF_F ? 0.f : mn;
        if (__any_sync(kFull, mn > m[i2])) {
          const float a = exp2f(m[i2] - mu[i2]);
          l[i2] *= a;
#pragma unroll
          for (int dt = 0; dt < DP / 8; ++dt) {
            o[dt][2 * i2] *= a;
            o[dt][2 * i2 + 1] *= a;
          }
        }
        m[i2] = mn;
      }
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[nt][e] = exp2f(s[nt][e] - mu[e >> 1]);
          l[e >> 1] += s[nt][e];
        }
      if (!F32) {
        uint32_t pa[4];
        pa[0] = pack_bf16(s[0][0], s[0][1]);
        pa[1] = pack_bf16(s[0][2], s[0][3]);
        pa[2] = pack_bf16(s[1][0], s[1][1]);
        pa[3] = pack_bf16(s[1][2], s[1][3]);
        const int vrow = lane & 15, vhalf = lane >> 4;
#pragma unroll
        for (int ds = 0; ds < DP / 16; ++ds) {
          uint32_t vb[4];
          ldmatrix_x4_trans(vb, sv + vrow * RB + (((2 * ds + vhalf) ^ (vrow & 7)) << 4));
          mma_bf16(o[2 * ds], pa, vb[0], vb[1]);
          mma_bf16(o[2 * ds + 1], pa, vb[2], vb[3]);
        }
      } else {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          // the score fragment's columns 2 t, 2 t + 1 serve as k = t, t + 4
          uint32_t ah[4], al[4];
          const int pick[4] = {0, 2, 1, 3};
#pragma unroll
          for (int e = 0; e < 4; ++e) split_tf32(s[nt][pick[e]], ah[e], al[e]);
#pragma unroll
          for (int dt = 0; dt < DP / 8; ++dt) {
            uint32_t bh[2], bl[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int key = nt * 8 + 2 * tq + e, d = dt * 8 + gr;
              const float x = *reinterpret_cast<const float*>(
                  sv_p + key * RB + (((d >> 2) ^ (key & 7)) << 4) + (d & 3) * 4);
              split_tf32(x, bh[e], bl[e]);
            }
            float part[4] = {};
            mma_tf32(part, al, bh[0], bh[1]);
            mma_tf32(part, ah, bl[0], bl[1]);
            mma_tf32(part, ah, bh[0], bh[1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[dt][e] += part[e];
          }
        }
      }
      __syncwarp();
      issue(i + S - 1, stage == 0 ? S - 1 : stage - 1);
      stage = stage + 1 == S ? 0 : stage + 1;
    }
    cp_async_wait<0>();
    // a row's sum over the four threads that hold its columns
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(kFull, l[i], 1);
      l[i] += __shfl_xor_sync(kFull, l[i], 2);
    }
    __syncthreads();
    // ---- join the four warps through shared memory (the rings are drained) ----
    constexpr int OP = DP + 4;  // padded output pitch
    float* so = reinterpret_cast<float*>(attn_dyn);            // [warp][16][OP]
    float* sm = so + kRowsWarps * kRowsR * OP;                 // [warp][16] m, then l
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = gr + 8 * i;
      if (tq == 0) {
        sm[warp * kRowsR + r] = m[i];
        sm[(kRowsWarps + warp) * kRowsR + r] = l[i];
      }
#pragma unroll
      for (int dt = 0; dt < DP / 8; ++dt)
        *reinterpret_cast<float2*>(so + (warp * kRowsR + r) * OP + dt * 8 + 2 * tq) =
            make_float2(o[dt][2 * i], o[dt][2 * i + 1]);
    }
    __syncthreads();
    constexpr int C = kRowsR * DP / kRowsThreads;  // columns of a thread
    const int r = threadIdx.x / (DP / C), c0 = (threadIdx.x % (DP / C)) * C;
    float mt = -CUDART_INF_F, lt = 0.f, ot[C];
#pragma unroll
    for (int w = 0; w < kRowsWarps; ++w) mt = fmaxf(mt, sm[w * kRowsR + r]);
    const float mbase = mt == -CUDART_INF_F ? 0.f : mt;
#pragma unroll
    for (int i = 0; i < C; ++i) ot[i] = 0.f;
#pragma unroll
    for (int w = 0; w < kRowsWarps; ++w) {
      const float mw = sm[w * kRowsR + r];
      const float a = exp2f(mw - mbase);
      lt += a * sm[(kRowsWarps + w) * kRowsR + r];
#pragma unroll
      for (int i = 0; i < C; ++i) ot[i] += a * so[(w * kRowsR + r) * OP + c0 + i];
    }
    if (F32) {
      bool odd = false;
#pragma unroll
      for (int i = 0; i < C; ++i) odd |= !(fabsf(ot[i]) < CUDART_INF_F);
      if (odd) take_nonfinite<C>(job, t, head, seg0, min(seg1, t.clear), c0, ot);
    }
    if (poison) {
      int b, n, g;
      if (attn_row(job, t, t.row0 + r, b, n, g))
        add_nonfinite<T, C>(job, t, head, n, max(t.clear, seg0), seg1, c0, ot);
    }
    if (SPLIT) {
      // the part of this CTA, then some columns of all of the cluster's parts
      float* po = sm + 2 * kRowsWarps * kRowsR;  // [16][OP], then [16] m and l
      float* pm = po + kRowsR * OP;
      if (c0 == 0) {
        pm[r] = mt;
        pm[kRowsR + r] = lt;
      }
#pragma unroll
      for (int i = 0; i < C; ++i) po[r * OP + c0 + i] = ot[i];
      cluster_barrier();
      const int rank = (int)cluster_rank(), size = (int)cluster_size();
      constexpr int UNITS = kRowsR * DP / 8;
      for (int u = UNITS / size * rank + threadIdx.x; u < UNITS / size * (rank + 1);
           u += kRowsThreads) {
        const int ur = u / (DP / 8), uc = (u % (DP / 8)) * 8;
        float m8 = -CUDART_INF_F, l8 = 0.f, o8[8] = {};
#pragma unroll 4
        for (int p = 0; p < size; ++p) {
          const float4 a = ld_cluster4(po + ur * OP + uc, p), b = ld_cluster4(po + ur * OP + uc + 4, p);
          const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
          join_part<8>(m8, l8, o8, ld_cluster(pm + ur, p), ld_cluster(pm + kRowsR + ur, p), x);
        }
        write_row<T, 8>(job, t, head, t.row0 + ur, uc, DP, m8, l8, o8);
      }
      cluster_barrier();  // the peers have read this CTA's part
      return;
    }
    if (nb == t.blocks) {
      write_row<T, C>(job, t, head, t.row0 + r, c0, DP, mt, lt, ot);
    } else {
      const int slot = 2 * cta + (block == 0 ? 1 : 0);
      if (c0 == 0) {
        job.part_ms[(slot * 2) * kRowsR + r] = mt;
        job.part_ms[(slot * 2 + 1) * kRowsR + r] = lt;
      }
      float4* dst = reinterpret_cast<float4*>(job.part_o + ((int64_t)slot * kRowsR + r) * DP + c0);
#pragma unroll
      for (int i = 0; i < C; i += 4)
        dst[i / 4] = make_float4(ot[i], ot[i + 1], ot[i + 2], ot[i + 3]);
      if (block == 0) {
        desc.x = 1;
        desc.y = head;
        desc.z = entry;
      } else {
        desc.w = block + nb == t.blocks ? kSlotEnd : kSlotMiddle;
      }
    }
    __syncthreads();
    if (threadIdx.x == 0) poison = 0;
    __syncthreads();
  }
  if (threadIdx.x == 0) job.part_desc[cta] = desc;
}

// ---------------------------------------------------------------------------------------
// Join of the tiles cut between CTAs.  Block (j, y) looks whether CTA j left a tile open and
// joins some rows of its parts: CTA j's second slot, then the first slots of the CTAs after
// it until the one that holds the tile's end.  A few rows of one long sequence leave a part in
// every CTA: with GROUPS > 1 the parts are dealt to that many groups of threads, each joining
// its own in the order of the keys, and the groups are joined through shared memory.
// ---------------------------------------------------------------------------------------

template <int DP, int R>
struct CombineCfg {
  static constexpr int kGroups = R == kRowsR ? 4 : 1;
  static constexpr int kGroupThreads = kCombineThreads / kGroups;
  static constexpr int kC = DP / 8;                 // columns of a thread
  static constexpr int kRows = kGroupThreads / 8;   // rows of a block
};

template <typename T, int DP, int R, int KB>
__global__ void __launch_bounds__(kCombineThreads) attn_combine_kernel(AttnJob job, int ctas) {
  using Cfg = CombineCfg<DP, R>;
  constexpr int GROUPS = Cfg::kGroups, GT = Cfg::kGroupThreads, C = Cfg::kC, BR = Cfg::kRows;
  constexpr int XG = GROUPS > 1 ? GROUPS - 1 : 1, XR = GROUPS > 1 ? BR : 1;
  __shared__ float s_ms[XG][XR][2];
  __shared__ float s_o[XG][XR][DP + 4];
  __shared__ int s_end;
  const int j = blockIdx.x;
  if (threadIdx.x == 0) s_end = ctas;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 desc = job.part_desc[j];
  if (!desc.x) return;
  __syncthreads();
  for (int i = j + 1 + threadIdx.x; i < ctas; i += kCombineThreads)
    if (job.part_desc[i].w == kSlotEnd) {
      atomicMin(&s_end, i);
      break;
    }
  const AttnTile t = attn_tile<R, KB>(job, desc.z);
  const int grp = threadIdx.x / GT, tg = threadIdx.x % GT;
  const int rr = tg / 8, r = blockIdx.y * BR + rr, c0 = (tg % 8) * C;
  __syncthreads();
  const int last = min(s_end, ctas - 1);  // its first slot holds the tile's end
  float m = -CUDART_INF_F, l = 0.f, o[C];
#pragma unroll
  for (int i = 0; i < C; ++i) o[i] = 0.f;
#pragma unroll 2
  for (int i = j + grp; i <= last; i += GROUPS) {
    const bool none = i > j && job.part_desc[i].w == kSlotNone;  // a CTA without work
    const int slot = i == j ? 2 * j + 1 : 2 * i;
    const float ms = none ? -CUDART_INF_F : job.part_ms[(slot * 2) * R + r];
    const float ls = none ? 0.f : job.part_ms[(slot * 2 + 1) * R + r];
    const float4* src =
        reinterpret_cast<const float4*>(job.part_o + ((int64_t)slot * R + r) * DP + c0);
    float x[C];
#pragma unroll
    for (int k = 0; k < C / 4; ++k) {
      const float4 v = none ? make_float4(0.f, 0.f, 0.f, 0.f) : src[k];
      x[4 * k] = v.x;
      x[4 * k + 1] = v.y;
      x[4 * k + 2] = v.z;
      x[4 * k + 3] = v.w;
    }
    join_part<C>(m, l, o, ms, ls, x);
  }
  if (GROUPS > 1) {
    if (grp > 0) {
      if (c0 == 0) {
        s_ms[grp - 1][rr][0] = m;
        s_ms[grp - 1][rr][1] = l;
      }
#pragma unroll
      for (int i = 0; i < C; ++i) s_o[grp - 1][rr][c0 + i] = o[i];
    }
    __syncthreads();
    if (grp > 0) return;
#pragma unroll
    for (int g = 0; g < GROUPS - 1; ++g) {
      float x[C];
#pragma unroll
      for (int i = 0; i < C; ++i) x[i] = s_o[g][rr][c0 + i];
      join_part<C>(m, l, o, s_ms[g][rr][0], s_ms[g][rr][1], x);
    }
  }
  write_row<T, C>(job, t, desc.y, t.row0 + r, c0, DP, m, l, o);
}

// The join starts while the attention kernel's last CTAs still run and waits for them
// (programmatic stream serialization).
template <typename T, int DP, int R, int KB>
cudaError_t launch_combine(const AttnJob& job, int ctas, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas, R / CombineCfg<DP, R>::kRows);
  cfg.blockDim = dim3(kCombineThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_combine_kernel<T, DP, R, KB>, job, ctas);
}

// Which cut: a tile to a cluster of up to eight CTAs where that many tiles' clusters are
// resident at once (with twice as many 11-node fp32 trees took 42 us instead of 35) and no CTA
// takes more than kSplitBlocks blocks even if the table's positions are all in use (the lengths
// are on the device).  Eight blocks are a middle of the types: one bf16 token on 3000 and 4000
// positions takes 12.8 and 14.4 us in clusters, 19.7 and 20.0 by the list, on 6000 17.5 and 21.9;
// 88 rows of fp32 on up to 2000 positions 29.0 and 24.6, on up to 3000 38.6 and 28.7.  Else the even work list, cut for the CTAs that are resident (cut for
// two or four times as many, so that a CTA that is done makes room for another, 64 requests of
// 4096 positions took 213 and 220 us instead of 204: the starts and the parts to join cost
// more than the even finish gives).  Returns the CTAs of a cluster, 0 for the list.
int64_t rows_tiles(const AttnJob& job) {
  const int64_t rows = job.phase == kShared ? (int64_t)job.B * job.N * job.G : (int64_t)job.N * job.G;
  return (rows + kRowsR - 1) / kRowsR * (job.phase == kShared ? 1 : job.B) * job.Hkv;
}
int rows_split(const AttnJob& job, int resident) {
  const int64_t tiles = rows_tiles(job);
  const int64_t positions = job.phase == kShared
                                ? job.shared_len
                                : (int64_t)job.max_pages * job.pd.size - job.shared_len;
  int split = kMaxSplit;
  while (split > 1 && tiles * split > resident) split /= 2;
  return (positions + kRowsKB - 1) / kRowsKB <= (int64_t)kSplitBlocks * split && tiles <= 0x7fffffff
             ? split
             : 0;
}
// bf16 calls whose rows the tensor-memory kernel could take, but which are one wave of
// clusters here: one short launch instead of a long one and a join.  One request of 1000 positions
// with 20 to 104 rows: 24 us a call instead of 27 to 30 (most of it the host's); 64 requests of
// 2000, which are no such wave: 208 to 782 us instead of 121 to 129.
bool rows_one_wave(const AttnJob& job) {
  const int resident = device_sm_count() * RowsCfg<uint16_t, 128>::kCtasPerSm;
  return rows_tiles(job) <= resident && rows_split(job, resident) > 0;
}

template <typename T, int DP>
cudaError_t launch_rows(AttnJob job, cudaStream_t s) {
  using Cfg = RowsCfg<T, DP>;
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    e = cudaFuncSetAttribute(attn_rows_kernel<T, DP, false>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(attn_rows_kernel<T, DP, true>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev] = true;
  }
  const int rows = job.phase == kShared ? job.B * job.N * job.G : job.N * job.G;
  job.row_tiles = (rows + kRowsR - 1) / kRowsR;
  job.entries = job.phase == kShared ? job.row_tiles : job.row_tiles * job.B;
  job.by_tiles = FastDiv::make(job.row_tiles);
  const int resident = device_sm_count() * Cfg::kCtasPerSm;
  const int split = rows_split(job, resident);
  if (split > 0) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(rows_tiles(job) * split));
    cfg.blockDim = dim3(kRowsThreads);
    cfg.dynamicSmemBytes = Cfg::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)split;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_rows_kernel<T, DP, true>, job);
  }
  const int grid = min(resident, kAttnMaxCtas);
  attn_rows_kernel<T, DP, false><<<grid, kRowsThreads, Cfg::kSmem, s>>>(job);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_combine<T, DP, kRowsR, kRowsKB>(job, grid, s);
}

// rows of all slots of a launch, whichever kernel it is
constexpr size_t kAttnSlotRows =
    2 * (size_t)(kAttnTcSlots > kAttnMaxCtas * kRowsR ? kAttnTcSlots : kAttnMaxCtas * kRowsR);

struct AttnWs {
  size_t desc, ms, o, own_lse, own_o, total;
};

int padded_dim(int d) { return d <= 64 ? 64 : 128; }

AttnWs attn_ws(int64_t rows, int Hq, int D, int shared_len) {
  AttnWs w{};
  const size_t DP = padded_dim(D);
  size_t off = 0;
  w.desc = off;
  off = align_up(off + kAttnMaxCtas * sizeof(int4), 256);
  w.ms = off;
  off = align_up(off + kAttnSlotRows * 2 * 4, 256);
  w.o = off;
  off = align_up(off + kAttnSlotRows * DP * 4, 256);
  w.own_lse = off;
  w.own_o = off;
  if (shared_len > 0) {
    off = align_up(off + (size_t)rows * Hq * 4, 256);
    w.own_o = off;
    off = align_up(off + (size_t)rows * Hq * DP * 4, 256);
  }
  w.total = off;
  return w;
}

}  // namespace

cudaError_t launch_attn_combine(const AttnJob& job, int DP, int R, int ctas, cudaStream_t s) {
  if (R == 256)
    return DP == 64 ? launch_combine<uint16_t, 64, 256, kAttnTcKeys>(job, ctas, s)
                    : launch_combine<uint16_t, 128, 256, kAttnTcKeys>(job, ctas, s);
  return DP == 64 ? launch_combine<uint16_t, 64, 128, kAttnTcKeys>(job, ctas, s)
                  : launch_combine<uint16_t, 128, 128, kAttnTcKeys>(job, ctas, s);
}

namespace {

bool attn_sizes_ok(int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t shared_len) {
  return B >= 0 && N >= 0 && Hq >= 1 && Hkv >= 1 && Hq % Hkv == 0 && D >= 1 && shared_len >= 0;
}

}  // namespace

}  // namespace svk

using namespace svk;

extern "C" size_t spec_tree_attention_workspace_size(int32_t B, int32_t N, int32_t n_q_heads,
                                                     int32_t n_kv_heads, int32_t head_dim,
                                                     int32_t shared_len, spec_dtype dtype) {
  if (!attn_sizes_ok(B, N, n_q_heads, n_kv_heads, head_dim, shared_len)) return 0;
  if (head_dim > SPEC_ATTN_MAX_HEAD_DIM || (int64_t)B * N * n_q_heads > 0x3fffffff ||
      shared_len > SPEC_MAX_POSITIONS)
    return 0;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return 0;
  return attn_ws((int64_t)B * N, n_q_heads, head_dim, shared_len).total;
}

extern "C" int spec_tree_attention_paged(
    const void* q, spec_node_layout q_layout, const void* k_cache, const void* v_cache,
    spec_paged_layout cache, spec_dtype dtype, int32_t B, int32_t N, int32_t n_q_heads,
    const int32_t* page_table, int32_t max_pages, const int32_t* prefix_len,
    const int32_t* counts, const uint8_t* mask, int32_t shared_len, float scale, void* out,
    spec_node_layout out_layout, float* lse, void* workspace, size_t workspace_bytes,
    spec_stream_t stream) {
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_UNSUPPORTED_DTYPE;
  int rc = check_paged_layout(cache, max_pages);
  if (rc != SPEC_OK) return rc;
  if (!attn_sizes_ok(B, N, n_q_heads, cache.n_kv_heads, cache.head_dim, shared_len) ||
      shared_len % cache.page_size != 0 || !(fabsf(scale) <= FLT_MAX))
    return SPEC_ERR_INVALID_ARG;
  // (the kernels add up to a few blocks to a position in 32 bits)
  if (cache.head_dim > SPEC_ATTN_MAX_HEAD_DIM || (int64_t)B * N * n_q_heads > 0x3fffffff ||
      shared_len > SPEC_MAX_POSITIONS)
    return SPEC_ERR_TOO_LARGE;
  if (B == 0 || N == 0) return SPEC_OK;
  if (!q || !k_cache || !v_cache || !page_table || !prefix_len || !out || !workspace)
    return SPEC_ERR_INVALID_ARG;
  const int64_t es = dtype == SPEC_F32 ? 4 : 2;
  const int64_t strides[] = {q_layout.batch_stride,   q_layout.node_stride,
                             q_layout.head_stride,    out_layout.batch_stride,
                             out_layout.node_stride,  out_layout.head_stride,
                             cache.page_stride,       cache.pos_stride,
                             cache.head_stride,       cache.head_dim};
  for (int64_t x : strides)
    if ((x * es) % 16 != 0) return SPEC_ERR_MISALIGNED;
  const void* bases[] = {q, k_cache, v_cache, out};
  for (const void* p : bases)
    if (reinterpret_cast<uintptr_t>(p) & 15u) return SPEC_ERR_MISALIGNED;
  const AttnWs w = attn_ws((int64_t)B * N, n_q_heads, cache.head_dim, shared_len);
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < w.total)
    return SPEC_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  AttnJob job{};
  job.q = q;
  job.k = k_cache;
  job.v = v_cache;
  job.out = out;
  job.lse = lse;
  job.lq = q_layout;
  job.lo = out_layout;
  job.page_stride = cache.page_stride;
  job.pos_stride = cache.pos_stride;
  job.head_stride = cache.head_stride;
  job.table = page_table;
  job.prefix = prefix_len;
  job.counts = counts;
  job.mask = mask;
  job.B = B;
  job.N = N;
  job.Hq = n_q_heads;
  job.Hkv = cache.n_kv_heads;
  job.G = n_q_heads / cache.n_kv_heads;
  job.D = cache.head_dim;
  job.n_pages = cache.n_pages;
  job.max_pages = max_pages;
  job.shared_len = shared_len;
  job.pd = PageDiv::make(cache.page_size);
  job.by_g = FastDiv::make(job.G);
  job.by_ng = FastDiv::make(N * job.G);
  job.scale_log2 = (float)((double)scale * 1.4426950408889634);
  job.part_desc = reinterpret_cast<int4*>(ws + w.desc);
  job.part_ms = reinterpret_cast<float*>(ws + w.ms);
  job.part_o = reinterpret_cast<float*>(ws + w.o);
  job.own_lse = reinterpret_cast<float*>(ws + w.own_lse);
  job.own_o = reinterpret_cast<float*>(ws + w.own_o);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool narrow = padded_dim(job.D) == 64;
  for (int phase = kOwn; phase <= (shared_len > 0 ? kShared : kOwn); ++phase) {
    job.phase = phase;
    cudaError_t e = cudaSuccess;
    bool taken = false;
    if (attn_tc_fits(job, dtype) && !rows_one_wave(job)) e = launch_attn_tc(job, s, &taken);
    if (e != cudaSuccess) return SPEC_ERR_CUDA;
    if (taken) continue;
    if (dtype == SPEC_BF16)
      e = narrow ? launch_rows<uint16_t, 64>(job, s) : launch_rows<uint16_t, 128>(job, s);
    else
      e = narrow ? launch_rows<float, 64>(job, s) : launch_rows<float, 128>(job, s);
    if (e != cudaSuccess) return SPEC_ERR_CUDA;
  }
  return SPEC_OK;
}
