// attention_tc.cu -- the many-rows kernel of the paged tree attention: bf16, tiles of 256
// rows on the fifth-generation tensor cores.
//
// A CTA holds the queries of two halves of 128 rows in shared memory and walks its tile's
// keys in blocks of 128:
//   warp 0      TMA producer: a block's keys and values, page by page (boxes of up to 128
//               rows that never cross a page), with the 128-byte swizzle into a ring
//   warp 1      MMA issuer: S_w = Q_w K^T (128 x 128, fp32 in tensor memory), then
//               O_w += P_w V with P_w read from tensor memory and V as it lies (its rows are
//               the product's inner direction)
//   warps 4-7   softmax of half 0, one row per thread: the row of S into registers, running
//   warps 8-11  maximum, exponentials, their sum, P back over S as bf16; half 1 likewise
// The halves take turns on the tensor cores: while one half's exponentials are formed the
// other half's products run.  The output stays in tensor memory and is scaled only when a
// row's maximum has risen by more than 2^8 since it was last scaled (the exponentials then
// stay below 2^8, far inside bf16's and fp32's range, and the quotient by their sum is the
// same), so the read-modify-write of the output is rare.
//
// Every wait is bounded; one that gives up sets a flag, all later waits return at once, the
// control flow runs to its end and the CTA's results become NaN.
#include "attention.cuh"
#include "tcgen05.cuh"

namespace svk {

namespace {

constexpr int kTcR = 256, kTcHalf = 128, kTcKB = 128;
constexpr int kTcThreads = 384;
constexpr uint32_t kTcTmemCols = 512;
constexpr float kTcLazy = 8.f;  // log2 of the rise that makes the output scaled

template <int DP>
struct TcCfg {
  static constexpr int kChunks = DP / 64;                  // 128-byte columns of a row
  static constexpr int kChunkBytes = 128 * 128;
  static constexpr int kStageBytes = kChunks * kChunkBytes; // 128 keys (or values)
  static constexpr int kQBytes = 2 * kStageBytes;
  static constexpr int kStages = DP == 64 ? 8 : 4;
  static constexpr int kSmem = 1024 + kQBytes + kStages * kStageBytes;
};

struct TcShared {
  uint64_t full[8], empty[8], q_full[2], s_full[2], p_full[2], o_full[2], done;
  uint32_t tmem;
  int abort;
  int poison;
};

struct TcWait {
  int* abort;
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) const {
    if (mbar_try(bar, parity)) return;
    const uint64_t t0 = global_ns();
    for (;;) {
      for (int k = 0; k < 32; ++k)
        if (mbar_try(bar, parity)) return;
      if (*((volatile int*)abort)) return;
      if (global_ns() - t0 > 2000000000ull) {
        *((volatile int*)abort) = 1;
        return;
      }
    }
  }
};


template <int DP>
__global__ void __launch_bounds__(kTcThreads, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ AttnJob job,
                   int box_rows) {
  using Cfg = TcCfg<DP>;
  constexpr int NST = Cfg::kStages;
  __shared__ TcShared sh;
  extern __shared__ unsigned char tc_dyn[];
  const uint32_t base = (smem_u32(tc_dyn) + 1023u) & ~1023u;
  unsigned char* base_p = tc_dyn + (base - smem_u32(tc_dyn));
  const uint32_t sq = base, ring = base + Cfg::kQBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&sh.q_full[w], kTcHalf);
      mbar_init(&sh.s_full[w], 1);
      mbar_init(&sh.p_full[w], kTcHalf);
      mbar_init(&sh.o_full[w], 1);
    }
    mbar_init(&sh.done, 1);
    sh.abort = 0;
    sh.poison = 0;
    fence_barrier_init();
  }
  if (warp == 1) tc05_alloc(&sh.tmem, kTcTmemCols);
  const AttnRange range = attn_range<kTcR, kTcKB, kTcThreads>(job, cta, gridDim.x);
  tc05_fence_before();
  __syncthreads();
  tc05_fence_after();
  const uint32_t tmem = sh.tmem;
  const TcWait wait{&sh.abort};
  const int rows_all = job.phase == kShared ? job.B * job.N * job.G : job.N * job.G;

  int64_t left = range.units;
  int head = range.head, entry = range.entry, block = range.block;
  uint32_t ent = 0;  // ring entries so far: key and value blocks in turn

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    const int boxes = kTcKB / box_rows;
    while (left > 0) {
      const AttnTile t = attn_tile<kTcR, kTcKB>(job, entry);
      const int nb = (int)min((int64_t)(t.blocks - block), left);
      const int32_t* table_row = job.table + (int64_t)t.b * job.max_pages;
      for (int i = 0; i < nb; ++i) {
        // a box with no page, or past the last visible key, is read outside the cache: zeros
        int page = job.n_pages, slot = 0;
        if (lane < boxes) {
          const int pos = t.kbeg + (block + i) * kTcKB + lane * box_rows;
          const int at = job.pd.div(pos);
          if (pos < t.kend && at < job.max_pages) {
            const int p = table_row[at];
            if ((unsigned)p < (unsigned)job.n_pages) {
              page = p;
              slot = pos - at * job.pd.size;
            }
          }
        }
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++ent) {
          const int s = (int)(ent % NST);
          wait(&sh.empty[s], ((ent / NST) & 1u) ^ 1u);
          if (lane == 0) mbar_arrive_expect_tx(&sh.full[s], Cfg::kStageBytes);
          __syncwarp();
          if (lane < boxes) {
            const uint32_t dst = ring + s * Cfg::kStageBytes + lane * box_rows * 128;
#pragma unroll
            for (int c = 0; c < Cfg::kChunks; ++c)
              tma_load_4d(dst + c * Cfg::kChunkBytes, kv ? &tm_v : &tm_k, c * 64, head, slot, page,
                          &sh.full[s]);
          }
        }
      }
      left -= nb;
      block = 0;
      if (++entry == job.entries) {
        entry = 0;
        ++head;
      }
    }
    // no copy may still be landing when the CTA exits
    const uint32_t first = ent > (uint32_t)NST ? ent - NST : 0u;
    for (uint32_t e = first; e < ent; ++e) wait(&sh.full[e % NST], (e / NST) & 1u);
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (lane == 0) {
      constexpr uint32_t idesc_s = bf16_idesc(kTcKB, false), idesc_o = bf16_idesc(DP, true);
      uint32_t seg[2] = {0, 0}, blk[2] = {0, 0};
      auto scores = [&](int w, uint32_t e) {
        const uint64_t a = sw128_tile(sq + w * Cfg::kStageBytes, 16);
        const uint64_t b = sw128_tile(ring + (e % NST) * Cfg::kStageBytes, 16);
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks) {
          const uint64_t off = (uint64_t)(((ks >> 2) * Cfg::kChunkBytes + (ks & 3) * 32) >> 4);
          tc05_mma_ss(tmem + w * 128, a + off, b + off, idesc_s, ks > 0);
        }
      };
      while (left > 0) {
        const AttnTile t = attn_tile<kTcR, kTcKB>(job, entry);
        const int nb = (int)min((int64_t)(t.blocks - block), left);
        const int halves = rows_all - t.row0 > kTcHalf ? 2 : 1;
        for (int w = 0; w < halves; ++w) wait(&sh.q_full[w], seg[w]++ & 1u);
        wait(&sh.full[ent % NST], (ent / NST) & 1u);
        tc05_fence_after();
        for (int w = 0; w < halves; ++w) {
          scores(w, ent);
          tc05_commit(&sh.s_full[w]);
        }
        tc05_commit(&sh.empty[ent % NST]);
        for (int i = 0; i < nb; ++i) {
          const uint32_t ev = ent + 2 * i + 1, ek = ev + 1;
          wait(&sh.full[ev % NST], (ev / NST) & 1u);
          for (int w = 0; w < halves; ++w) {
            wait(&sh.p_full[w], blk[w]++ & 1u);
            tc05_fence_after();
            const uint64_t b = sw128_tile(ring + (ev % NST) * Cfg::kStageBytes, Cfg::kChunkBytes);
#pragma unroll
            for (int ks = 0; ks < kTcKB / 16; ++ks)
              tc05_mma_ts(tmem + 256 + w * 128, tmem + w * 128 + ks * 8,
                          b + (uint64_t)((ks * 2048) >> 4), idesc_o, i > 0 || ks > 0);
            if (w == halves - 1) tc05_commit(&sh.empty[ev % NST]);
            if (i + 1 < nb) {
              if (w == 0) {
                wait(&sh.full[ek % NST], (ek / NST) & 1u);
                tc05_fence_after();
              }
              scores(w, ek);
              tc05_commit(&sh.s_full[w]);
              if (w == halves - 1) tc05_commit(&sh.empty[ek % NST]);
            } else {
              tc05_commit(&sh.o_full[w]);
            }
          }
        }
        ent += 2 * nb;
        left -= nb;
        block = 0;
        if (++entry == job.entries) {
          entry = 0;
          ++head;
        }
      }
      tc05_commit(&sh.done);
      wait(&sh.done, 0u);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---------------- softmax and epilogue of one half ----------------
    const int w = (warp - 4) >> 2;
    const int tid = (int)threadIdx.x - 128 - w * 128;  // 0 .. 127: the row within the half
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t t_s = lanes + w * 128, t_o = lanes + 256 + w * 128;
    const float c = fabsf(job.scale_log2);
    const uint32_t flip = job.scale_log2 < 0.f ? 0x80008000u : 0u;  // the maximum wants c >= 0
    const int boxes = kTcKB / box_rows, box_shift = 31 - __clz(box_rows);
    uint32_t seg = 0, blk = 0;

    // the half's queries into shared memory (K-major, 128-byte swizzle)
    auto load_q = [&](int hd, int en) {
      const AttnTile t = attn_tile<kTcR, kTcKB>(job, en);
      if (w == 1 && rows_all - t.row0 <= kTcHalf) return;
      constexpr int CPR = DP / 8;  // 16-byte units of a row
      const int u = tid % CPR;
      unsigned char* dst = base_p + w * Cfg::kStageBytes + (u >> 3) * Cfg::kChunkBytes;
      constexpr int kBatch = 8;
      for (int r0 = tid / CPR; r0 < kTcHalf; r0 += kBatch * (kTcHalf / CPR)) {
        uint4 x[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int r = r0 + i * (kTcHalf / CPR);
          x[i] = make_uint4(0, 0, 0, 0);
          int b, node, g;
          if (r < kTcHalf && attn_row(job, t, t.row0 + w * kTcHalf + r, b, node, g) &&
              u * 8 < job.D)
            x[i] = *reinterpret_cast<const uint4*>(
                static_cast<const uint16_t*>(job.q) + b * job.lq.batch_stride +
                node * job.lq.node_stride + (hd * job.G + g) * job.lq.head_stride + u * 8);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int r = r0 + i * (kTcHalf / CPR);
          if (r >= kTcHalf) break;
          x[i].x ^= flip;
          x[i].y ^= flip;
          x[i].z ^= flip;
          x[i].w ^= flip;
          *reinterpret_cast<uint4*>(dst + r * 128 + (((u & 7) ^ (r & 7)) << 4)) = x[i];
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&sh.q_full[w]);
    };
    if (left > 0) load_q(head, entry);
    int4 desc = make_int4(0, 0, 0, kSlotNone);
    while (left > 0) {
      const AttnTile t = attn_tile<kTcR, kTcKB>(job, entry);
      const int nb = (int)min((int64_t)(t.blocks - block), left);
      const int halves = rows_all - t.row0 > kTcHalf ? 2 : 1;
      int next_head = head, next_entry = entry + 1;
      if (next_entry == job.entries) {
        next_entry = 0;
        ++next_head;
      }
      const int seg0 = t.kbeg + block * kTcKB;
      if (w < halves) {
        const int r = t.row0 + w * kTcHalf + tid;
        int rb, node, g;
        const bool real = attn_row(job, t, r, rb, node, g);
        const int32_t* table_row = job.table + (int64_t)t.b * job.max_pages;
        float m = -CUDART_INF_F, l = 0.f;
        // page of this lane's box of the next block
        auto box_ok = [&](int i) {
          const int pos = seg0 + i * kTcKB + lane * box_rows;
          if (lane >= boxes || pos >= t.kend) return true;  // past the end: masked there
          const int at = job.pd.div(pos);
          return at < job.max_pages && (unsigned)table_row[at] < (unsigned)job.n_pages;
        };
        bool ok_next = box_ok(0);
        for (int i = 0; i < nb; ++i) {
          const int pos0 = seg0 + i * kTcKB;
          const unsigned ok = __ballot_sync(kFull, ok_next);
          if (i + 1 < nb) ok_next = box_ok(i + 1);
          const bool drafts = pos0 + kTcKB > min(t.prefix, t.kend);  // rows may differ in what they see
          uint32_t sees[4];
          if (drafts || ok != kFull) {
            // bit k of word j: this row sees key 32 j + k of the block
            const int lim = min(t.prefix, t.kend) - pos0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int n = min(max(lim - 32 * j, 0), 32);
              sees[j] = n == 32 ? kFull : (1u << n) - 1u;
            }
            if (drafts && job.phase == kOwn && real && node < t.count) {
              const int from = max(pos0, t.prefix), to = min(pos0 + kTcKB, t.kend);
              if (!job.mask) {
                const int end = min(to - t.prefix, node + 1) + (t.prefix - pos0);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const int n = min(max(end - 32 * j, 0), 32);
                  sees[j] = n == 32 ? kFull : (1u << n) - 1u;
                }
              } else {
                const uint8_t* mrow = job.mask + ((int64_t)t.b * job.N + node) * job.N - t.prefix;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const int lo = max(from, pos0 + 32 * j), hi = min(to, pos0 + 32 * j + 32);
                  for (int p = lo; p < hi; ++p)
                    if (mrow[p]) sees[j] |= 1u << (p - pos0 - 32 * j);
                }
              }
            }
            if (ok != kFull) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                for (int k = 0; k < 32; k += 8)
                  if (!((ok >> ((32 * j + k) >> box_shift)) & 1u)) sees[j] &= ~(0xffu << k);
            }
          }
          wait(&sh.s_full[w], blk & 1u);
          ++blk;
          __syncwarp();
          tc05_fence_after();
          uint32_t s[128];
          tc05_ld32(t_s, s);
          tc05_ld32(t_s + 32, s + 32);
          tc05_ld32(t_s + 64, s + 64);
          tc05_ld32(t_s + 96, s + 96);
          tc05_wait_ld();
          tc05_landed(s);
          tc05_landed(s + 32);
          tc05_landed(s + 64);
          tc05_landed(s + 96);
          if (drafts || ok != kFull) {
#pragma unroll
            for (int k = 0; k < 128; ++k)
              if (!((sees[k >> 5] >> (k & 31)) & 1u)) s[k] = 0xff800000u;  // -inf
          }
          float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
          for (int k = 0; k < 128; k += 8)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              mx[q] = fmaxf(mx[q], fmaxf(__uint_as_float(s[k + 2 * q]), __uint_as_float(s[k + 2 * q + 1])));
          const float mn = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), m);
          const bool rise = mn > m && (m == -CUDART_INF_F || (mn - m) * c > kTcLazy);
          if (__any_sync(kFull, rise)) {
            const float a = (rise && m != -CUDART_INF_F) ? ex2_approx((m - mn) * c)
                            : (rise ? 0.f : 1.f);
            if (i > 0) {
#pragma unroll 1
              for (int ch = 0; ch < DP; ch += 16) {
                uint32_t o[16];
                tc05_ld16(t_o + ch, o);
                tc05_wait_ld();
                tc05_landed16(o);
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
                tc05_st16(t_o + ch, o);
              }
            }
            l *= a;
            if (rise) m = mn;
          }
          const float mc = m == -CUDART_INF_F ? 0.f : m * c;
          const float2 c2 = make_float2(c, c), n2 = make_float2(-mc, -mc);
          float2 sum = make_float2(0.f, 0.f), sum2 = sum;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t p[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const int e = 64 * half + 2 * k;
              float2 x = fma_f32x2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])),
                                   c2, n2);
              x.x = ex2_approx(x.x);
              x.y = ex2_approx(x.y);
              if (k & 1) sum = add_f32x2(sum, x);
              else sum2 = add_f32x2(sum2, x);
              p[k] = pack_bf16(x.x, x.y);
            }
            tc05_st32(t_s + 32 * half, p);
          }
          sum = add_f32x2(sum, sum2);
          l += sum.x + sum.y;
          if (drafts) {
            // values past the last visible key leave the product, and so do infinities and
            // NaN among the drafts (a row that does not see them has weight 0 for them)
            const uint32_t ev = ent + 2 * i + 1;
            wait(&sh.full[ev % NST], (ev / NST) & 1u);
            constexpr int CPR = DP / 8;
            const int k0 = max(t.prefix - pos0, 0), kn = t.kend - pos0;
            unsigned char* vb = base_p + Cfg::kQBytes + (ev % NST) * Cfg::kStageBytes;
            for (int x = k0 * CPR + w * kTcHalf + tid; x < kTcKB * CPR; x += halves * kTcHalf) {
              const int key = x / CPR, u = x % CPR;
              uint4* at = reinterpret_cast<uint4*>(vb + (u >> 3) * Cfg::kChunkBytes + key * 128 +
                                                   (((u & 7) ^ (key & 7)) << 4));
              if (key >= kn) {
                *at = make_uint4(0, 0, 0, 0);
              } else {
                const uint4 v = *at;
                if (unit_nonfinite<uint16_t>(v)) {
                  uint32_t z[4] = {v.x, v.y, v.z, v.w};
                  for (int e = 0; e < 4; ++e) {
                    if ((z[e] & 0x7f800000u) == 0x7f800000u) z[e] &= 0xffffu;
                    if ((z[e] & 0x7f80u) == 0x7f80u) z[e] &= 0xffff0000u;
                  }
                  *at = make_uint4(z[0], z[1], z[2], z[3]);
                  *((volatile int*)&sh.poison) = 1;
                }
              }
            }
            fence_proxy_async_smem();
            asm volatile("bar.sync 2, %0;\n" ::"r"(halves * kTcHalf) : "memory");
          }
          __syncwarp();
          tc05_wait_st();
          tc05_fence_before();
          mbar_arrive(&sh.p_full[w]);
        }
        // the last scores are read: the half's queries may be replaced
        if (left > nb) load_q(next_head, next_entry);
        wait(&sh.o_full[w], seg & 1u);
        ++seg;
        __syncwarp();
        tc05_fence_after();
        if (*((volatile int*)&sh.abort)) l = __int_as_float(0x7fc00000);
        const float m2 = m == -CUDART_INF_F ? m : m * c;
        const bool whole = nb == t.blocks;
        const int slot = 2 * cta + (block == 0 ? 1 : 0);
        const int seg1 = min(seg0 + nb * kTcKB, t.kend);
        const bool poisoned = *((volatile int*)&sh.poison) != 0;
#pragma unroll 1
        for (int ch = 0; ch < DP; ch += 32) {
          uint32_t o[32];
          __syncwarp();
          tc05_ld32(t_o + ch, o);
          tc05_wait_ld();
          tc05_landed(o);
          float of[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) of[k] = __uint_as_float(o[k]);
          if (poisoned && job.phase == kOwn && real)
            add_nonfinite<uint16_t, 32>(job, t, head, node, max(t.prefix, seg0), seg1, ch, of);
          if (whole) {
            write_row<uint16_t, 32>(job, t, head, r, ch, DP, m2, l, of);
          } else {
            const int rr = r - t.row0;
            float4* dst =
                reinterpret_cast<float4*>(job.part_o + ((int64_t)slot * kTcR + rr) * DP + ch);
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              dst[k / 4] = make_float4(of[k], of[k + 1], of[k + 2], of[k + 3]);
            if (ch == 0) {
              job.part_ms[(slot * 2) * kTcR + rr] = m2;
              job.part_ms[(slot * 2 + 1) * kTcR + rr] = l;
            }
          }
        }
        tc05_fence_before();
      } else if (left > nb) {
        load_q(next_head, next_entry);  // this half idles in this tile
      }
      if (nb != t.blocks) {
        if (block == 0) {
          desc.x = 1;
          desc.y = head;
          desc.z = entry;
        } else {
          desc.w = block + nb == t.blocks ? kSlotEnd : kSlotMiddle;
        }
      }
      ent += 2 * nb;
      left -= nb;
      block = 0;
      head = next_head;
      entry = next_entry;
    }
    if (threadIdx.x == 128) job.part_desc[cta] = desc;
  }
  tc05_fence_before();
  __syncthreads();
  tc05_fence_after();
  if (warp == 1) tc05_dealloc(tmem, kTcTmemCols);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  }
  return fn;
}

// Rows of a box: the largest power of two that divides the page length, at most a block.
int tc_box_rows(int page_size) {
  const int low = page_size & -page_size;
  return low < kTcKB ? low : kTcKB;
}

// [page][slot][head][d] as a 4-D tensor; a box is 64 d of one head in box_rows slots of a page.
bool make_cache_map(CUtensorMap* map, const void* ptr, const AttnJob& job, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)job.D, (cuuint64_t)job.Hkv, (cuuint64_t)job.pd.size,
                              (cuuint64_t)job.n_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)job.head_stride * 2, (cuuint64_t)job.pos_stride * 2,
                                 (cuuint64_t)job.page_stride * 2};
  const cuuint32_t box[4] = {64, 1, (cuuint32_t)box_rows, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DP>
cudaError_t launch_tc(AttnJob job, cudaStream_t s, bool* taken) {
  using Cfg = TcCfg<DP>;
  const int box = tc_box_rows(job.pd.size);
  CUtensorMap tm_k, tm_v;
  *taken = make_cache_map(&tm_k, job.k, job, box) && make_cache_map(&tm_v, job.v, job, box);
  if (!*taken) return cudaSuccess;
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    e = cudaFuncSetAttribute(attn_tc_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Cfg::kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev] = true;
  }
  const int rows = job.phase == kShared ? job.B * job.N * job.G : job.N * job.G;
  job.row_tiles = (rows + kTcR - 1) / kTcR;
  job.entries = job.phase == kShared ? job.row_tiles : job.row_tiles * job.B;
  const int sms = device_sm_count();
  const int grid = sms < kAttnTcCtas ? sms : kAttnTcCtas;
  attn_tc_kernel<DP><<<grid, kTcThreads, Cfg::kSmem, s>>>(tm_k, tm_v, job, box);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_attn_combine(job, DP, kTcR, kTcKB, grid, s);
}

}  // namespace

// Few rows do not pay for 128-row products, and a box of fewer than 8 rows does not fill a
// swizzle group.
bool attn_tc_fits(const AttnJob& job, spec_dtype dtype) {
  const int64_t rows = job.phase == kShared ? (int64_t)job.B * job.N * job.G : (int64_t)job.N * job.G;
  return dtype == SPEC_BF16 && job.pd.size % 8 == 0 && job.n_pages > 0 && rows > kAttnRowsTile;
}

cudaError_t launch_attn_tc(const AttnJob& job, cudaStream_t s, bool* taken) {
  return job.D <= 64 ? launch_tc<64>(job, s, taken) : launch_tc<128>(job, s, taken);
}

}  // namespace svk
