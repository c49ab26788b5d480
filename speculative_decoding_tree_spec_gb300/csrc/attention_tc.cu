// attention_tc.cu -- the many-rows kernel of the paged tree attention: bf16, tiles of 256
// rows (or 128) on the fifth-generation tensor cores.
//
// A CTA holds the queries of one or two halves of 128 rows in shared memory and walks its
// tile's keys in blocks of 128:
//   warp 0      TMA producer: a block's keys and values, page by page (boxes of up to 128
//               rows that never cross a page), with the 128-byte swizzle into a ring
//   warp 1      MMA issuer: S_w = Q_w K^T (128 x 128, fp32 in tensor memory), then
//               O_w += P_w V with P_w read from tensor memory and V as it lies (its rows are
//               the product's inner direction)
//   warps 2-5   softmax of half 0, one row per thread: the row of S into registers, running
//   warps 6-9   maximum, exponentials, their sum, P back over S as bf16; half 1 likewise
// The halves take turns on the tensor cores: while one half's exponentials are formed the
// other half's products run.  P goes out in two parts of 64 keys, so that the first part's
// product runs while the second part's exponentials are formed.
// The 128 scores of a row are read once for the maximum; the upper 64 stay in registers and
// P goes over their place, so that the lower 64 can be read a second time and no thread needs
// more than about 128 registers for them.
// (Blocks of 64 keys with two score buffers per half, which take the scores off that chain,
// were slower: a 128 x 64 product takes the tensor cores as long as a 128 x 128 one.  A fixed
// reference in the maximum's place was no faster, a part of the exponentials by polynomial
// slower.  What bounds the kernel is latency in that chain: with two softmax warps per
// scheduler, each thread alone with its row, the issue slots are 33 % and the tensor pipe 45 %
// active (6656 rows of 4096 positions).  26624 rows of 8192 shared positions, 893 GFLOP: 703 us
// with the join of the own part, 1270 TFLOP/s, 68 % of the measured rate.)
// The output stays in tensor memory and is scaled only when a row's maximum has risen by more
// than 2^8 since it was last scaled (the exponentials then stay below 2^8, far inside bf16's
// and fp32's range, and the quotient by their sum is the same), so the read-modify-write of
// the output is rare.
//
// Every wait is bounded; one that gives up sets a flag, all later waits return at once, the
// control flow runs to its end and the CTA's results become NaN.
#include "attention.cuh"
#include "tcgen05.cuh"
#include "tensormap.cuh"

namespace svk {

namespace {

constexpr int kTcHalf = 128, kTcKB = kAttnTcKeys;
// A tile's fixed costs in blocks.  With 2, 3, 4 and 6 two 4096-token prompts take 316, 297, 279
// and 273 us (their tiles' lengths differ most), 64 trees of 240 rows on 512 to 4096 positions
// 182, 181, 179 and 178, of 80 rows on 2000 positions 118, 118, 118 and 120; 26624 rows of shared
// positions 863, 865, 856 and 858 with their own part.
constexpr int kTcC = 6;
constexpr uint32_t kTcP = 64;      // P's column within a half's scores
constexpr int kTcStagePitch = 80;  // bytes of a staged row: 64 and a pad against bank conflicts
constexpr int kTcCheck = 4;        // blocks whose page numbers are checked at once
constexpr uint64_t kTcLimitNs = 2000000000ull;  // of a wait
constexpr float kTcLazy = 8.f;     // log2 of the rise that makes the output scaled

// H halves of 128 rows in a tile.  H = 2: one CTA per SM.  H = 1 (tiles of at most 128 rows):
// two CTAs per SM, each with half of the tensor memory, whose loads, products and epilogues
// overlap each other's: 64 trees of 20 to 128 rows on 2000 positions take 121 to 129 us, with
// H = 2 141 to 148.  With more rows the second tile reads the keys again: 64 trees of 132, 240, 400
// and 512 rows on 2000 positions take 154, 173, 315 and 322 us with H = 2, 206, 221, 409 and 420
// with H = 1 (just above 256 rows, where H = 2 has a second tile for 4 rows, 296 against 307).
template <int DP, int H>
struct TcCfg {
  static constexpr int kR = kTcHalf * H;
  static constexpr int kThreads = 64 + kTcHalf * H;
  static constexpr uint32_t kTmemCols = 256 * H;            // per half: scores, output
  static constexpr int kChunks = DP / 64;                   // 128-byte columns of a row
  static constexpr int kQChunkBytes = kTcHalf * 128;
  static constexpr int kQHalfBytes = kChunks * kQChunkBytes;
  static constexpr int kQBytes = H * kQHalfBytes;
  static constexpr int kChunkBytes = kTcKB * 128;
  static constexpr int kStageBytes = kChunks * kChunkBytes; // 128 keys (or values)
  static constexpr int kStages = (DP == 64 ? 4 : 2) * H;
  static constexpr int kStaging = 4 * H * kTcStagePitch * 32;  // a warp's 32 rows of 64 bytes
  static constexpr int kSmem = 1024 + kQBytes + kStages * kStageBytes + kStaging;
};

struct TcShared {
  uint64_t full[8], empty[8];  // ring entries: key and value blocks in turn
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2][2], o_full[2], done;
  uint32_t tmem;
  int abort;
  int poison;
};

struct TcWait {
  int* abort;
  __device__ __forceinline__ bool aborted() const { return *((volatile int*)abort) != 0; }
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) const {
    // the clock is read after many tries only: a read takes longer than most waits
    uint64_t t0 = 0;
    for (uint32_t tries = 1;; ++tries) {
      if (mbar_try(bar, parity)) return;
      if ((tries & 1023u) == 0) {
        if (aborted()) return;
        const uint64_t now = global_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > kTcLimitNs) {
          *((volatile int*)abort) = 1;
          return;
        }
      }
    }
  }
};

// The softmax warps of a tile's halves meet.  A number for each count of threads: after a wait that
// gave up, a half may be in a later tile than the other.
template <int NUMBER, int THREADS>
__device__ __forceinline__ void half_barrier() {
  asm volatile("bar.sync %0, %1;\n" ::"n"(NUMBER), "n"(THREADS) : "memory");
}

template <int DP, int H>
__global__ void __launch_bounds__(TcCfg<DP, H>::kThreads, 3 - H)
    attn_tc_kernel(const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ AttnJob job,
                   int box_rows) {
  using Cfg = TcCfg<DP, H>;
  constexpr int kTcR = Cfg::kR;
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
      mbar_init(&sh.q_full[w], job.q_tma ? 1 : 4);
      mbar_init(&sh.q_empty[w], 1);
      mbar_init(&sh.s_full[w], 1);
      mbar_init(&sh.p_full[w][0], 4);
      mbar_init(&sh.p_full[w][1], 4);
      mbar_init(&sh.o_full[w], 1);
    }
    mbar_init(&sh.done, 1);
    sh.abort = 0;
    sh.poison = 0;
    fence_barrier_init();
  }
  if (warp == 1) tc05_alloc(&sh.tmem, Cfg::kTmemCols);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may line up
  const AttnRange range = attn_range<kTcR, kTcKB, kTcC, Cfg::kThreads>(job, cta, gridDim.x);
  tc05_fence_before();
  __syncthreads();
  tc05_fence_after();
  const uint32_t tmem = sh.tmem;
  const TcWait wait{&sh.abort};
  const int rows_all = job.phase == kShared ? job.B * job.N * job.G : job.N * job.G;

  AttnWalk<kTcC> walk(range);
  uint32_t ent = 0;  // ring entries so far: key and value blocks in turn

  AttnLens lens = attn_lens(job, walk.entry);  // read a tile ahead from here on
  if (warp == 0) {
    // ---------------- TMA producer ----------------
    const int boxes = kTcKB / box_rows;
    uint32_t q_loads[H] = {};
    for (; walk.left > 0; walk.next(job)) {
      const AttnTile t = attn_tile<kTcR, kTcKB>(job, walk.entry, lens);
      lens = attn_lens(job, walk.next_entry(job));
      walk.take(t.blocks);
      const int nb = walk.blocks, head = walk.head;
      const int32_t* table_row = job.table + (int64_t)t.b * job.max_pages;
      const int pos0 = t.kbeg + walk.first * kTcKB + lane * box_rows;  // this lane's box of block 0
      auto page_of = [&](int i) {
        const int pos = pos0 + i * kTcKB;
        return lane < boxes && i < nb && pos < t.kend ? table_row[job.pd.div(pos)] : -1;
      };
      // one box of each 64 columns; a box with no page, or past the last visible key, is read
      // outside the cache: zeros
      auto issue = [&](const CUtensorMap* tm, int page, int i) {
        const int s = (int)(ent % NST);
        wait(&sh.empty[s], ((ent / NST) & 1u) ^ 1u);
        if (__any_sync(kFull, wait.aborted())) return;  // the stage may still be in use
        if (lane == 0) mbar_arrive_expect_tx(&sh.full[s], Cfg::kStageBytes);
        __syncwarp();
        if (lane < boxes) {
          const int pos = pos0 + i * kTcKB;
          const bool there = (unsigned)page < (unsigned)job.n_pages;
          const int slot = there ? pos - job.pd.div(pos) * job.pd.size : 0;
          const uint32_t dst = ring + s * Cfg::kStageBytes + lane * box_rows * 128;
#pragma unroll
          for (int c = 0; c < Cfg::kChunks; ++c)
            tma_load_4d(dst + c * Cfg::kChunkBytes, tm, c * 64, head, slot,
                        there ? page : job.n_pages, &sh.full[s]);
        }
        ++ent;
      };
      int page = page_of(0);
      for (int i = 0; i < nb; ++i) {
        const int next = page_of(i + 1);
        issue(&tm_k, page, i);
        if (i == 0 && job.q_tma) {
          // the tile's queries, once the scores of the tile before have read theirs: rows
          // (node, query head of the key head) of each half
#pragma unroll
          for (int w = 0; w < H; ++w) {
            if (rows_all - t.row0 <= w * kTcHalf) break;
            wait(&sh.q_empty[w], (q_loads[w]++ & 1u) ^ 1u);
            if (__any_sync(kFull, wait.aborted())) break;
            if (lane == 0) {
              mbar_arrive_expect_tx(&sh.q_full[w], Cfg::kQHalfBytes);
#pragma unroll
              for (int c = 0; c < Cfg::kChunks; ++c)
                tma_load_4d(sq + w * Cfg::kQHalfBytes + c * Cfg::kQChunkBytes, &tm_q, c * 64,
                            head * job.G, job.by_g.div(t.row0 + w * kTcHalf), t.b, &sh.q_full[w]);
            }
            __syncwarp();
          }
        }
        issue(&tm_v, page, i);
        page = next;
      }
    }
    // no copy may still be landing when the CTA exits
    const uint32_t first = ent > (uint32_t)NST ? ent - NST : 0u;
    for (uint32_t e = first; e < ent; ++e)
      mbar_wait(&sh.full[e % NST], (e / NST) & 1u, kTcLimitNs);
#pragma unroll
    for (int w = 0; w < H; ++w)
      if (q_loads[w] > 0) mbar_wait(&sh.q_full[w], (q_loads[w] - 1) & 1u, kTcLimitNs);
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    constexpr uint32_t idesc_s = bf16_idesc(kTcKB, false), idesc_o = bf16_idesc(DP, true);
    uint32_t seg[H] = {}, blk[H] = {};
    auto scores = [&](int w, uint32_t stage, bool last) {  // last: of the tile
      const uint64_t a = sw128_tile(sq + w * Cfg::kQHalfBytes, 16);
      const uint64_t b = sw128_tile(ring + stage * Cfg::kStageBytes, 16);
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks)
          tc05_mma_ss(tmem + w * 256,
                      a + (uint64_t)(((ks >> 2) * Cfg::kQChunkBytes + (ks & 3) * 32) >> 4),
                      b + (uint64_t)(((ks >> 2) * Cfg::kChunkBytes + (ks & 3) * 32) >> 4), idesc_s,
                      ks > 0);
        tc05_commit(&sh.s_full[w]);
        if (last) tc05_commit(&sh.q_empty[w]);
      }
      __syncwarp();
    };
    auto release = [&](uint32_t stage) {
      if (elect_one()) tc05_commit(&sh.empty[stage]);
      __syncwarp();
    };
    // the ring's position: stage of the next entry and its barrier's parity
    uint32_t st = 0, par = 0;
    auto advance = [&]() {
      if (++st == (uint32_t)NST) {
        st = 0;
        par ^= 1u;
      }
    };
    // (after a wait that gave up the products run on whatever the buffers hold, within their
    // bounds)
    for (; walk.left > 0; walk.next(job)) {
      const AttnTile t = attn_tile<kTcR, kTcKB>(job, walk.entry, lens);
      lens = attn_lens(job, walk.next_entry(job));
      walk.take(t.blocks);
      const int nb = uniform(walk.blocks);
      const int halves = uniform(H == 2 && rows_all - t.row0 > kTcHalf ? 2 : 1);
#pragma unroll
      for (int w = 0; w < H; ++w)
        if (w < halves) wait(&sh.q_full[w], seg[w]++ & 1u);
      wait(&sh.full[st], par);
      tc05_fence_after();
#pragma unroll
      for (int w = 0; w < H; ++w)
        if (w < halves) scores(w, st, nb == 1);
      release(st);
      advance();
      for (int i = 0; i < nb; ++i) {
        const bool more = i + 1 < nb;
        const uint32_t sv = st, pv = par;  // V_i; K_{i+1} follows it
        advance();
        const uint32_t sk = st, pk = par;
        if (more) advance();
        wait(&sh.full[sv], pv);
#pragma unroll
        for (int w = 0; w < H; ++w) {
          if (w >= halves) break;
          const uint32_t parity = blk[w]++ & 1u;
          const uint64_t b = sw128_tile(ring + sv * Cfg::kStageBytes, Cfg::kChunkBytes);
          // keys 64 .. 127 first: their exponentials are
#pragma unroll
          for (int part = 1; part >= 0; --part) {
            wait(&sh.p_full[w][part], parity);
            tc05_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int ks = 4 * part; ks < 4 * part + 4; ++ks)
                tc05_mma_ts(tmem + w * 256 + 128, tmem + w * 256 + kTcP + ks * 8,
                            b + (uint64_t)((ks * 2048) >> 4), idesc_o,
                            i > 0 || part == 0 || ks > 4);
              if (part == 0 && !more) tc05_commit(&sh.o_full[w]);
            }
            __syncwarp();
          }
          if (w == halves - 1) release(sv);
          if (more) {
            if (w == 0) {
              wait(&sh.full[sk], pk);
              tc05_fence_after();
            }
            scores(w, sk, i + 2 == nb);
            if (w == halves - 1) release(sk);
          }
        }
      }
    }
    // every product issued has finished before the tensor memory is freed
    if (elect_one()) tc05_commit(&sh.done);
    __syncwarp();
    mbar_wait(&sh.done, 0u, kTcLimitNs);
    __syncwarp();
  } else {
    // ---------------- softmax and epilogue of one half ----------------
    // A warp's tensor-memory lanes are 32 (warp % 4) .. + 31: rows of the half by that number.
    const int w = (warp - 2) >> 2;
    const int tid = (warp & 3) * 32 + lane;  // 0 .. 127: the row within the half
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t t_s = lanes + w * 256, t_o = t_s + 128;
    const float c = job.scale_log2;  // > 0: maximum and mask stand before the scaling
    const int boxes = kTcKB / box_rows, box_shift = 31 - __clz(box_rows);
    uint32_t blk = 0, seg = 0;  // blocks and segments of this half so far

    // Where no tensor map takes them: the half's queries into shared memory (K-major, 128-byte
    // swizzle), each warp its 32 rows, a few rows to a copy; landed_q, later, hands them to the
    // products.
    auto load_q = [&](int hd, const AttnTile& t) {
      if (job.q_tma) return;
      if (H == 2 && w == 1 && rows_all - t.row0 <= kTcHalf) return;
      int b, node, g;
      const bool real = attn_row(job, t, t.row0 + w * kTcHalf + tid, b, node, g);
      const int64_t mine = real ? b * job.lq.batch_stride + node * job.lq.node_stride +
                                      (hd * job.G + g) * job.lq.head_stride
                                : (int64_t)-1;
      constexpr int CPR = DP / 8, STEP = 32 / CPR;  // 16-byte units of a row; rows of a step
      const int u = lane % CPR, r0 = lane / CPR;
      const uint32_t dst = sq + w * Cfg::kQHalfBytes + (u >> 3) * Cfg::kQChunkBytes;
#pragma unroll 4
      for (int i = 0; i < CPR; ++i) {
        const int64_t at = __shfl_sync(kFull, mine, r0 + i * STEP);
        const int r = (warp & 3) * 32 + r0 + i * STEP;
        const bool there = at >= 0 && u * 8 < job.D;
        cp_async16_or_zero(dst + r * 128 + (((u & 7) ^ (r & 7)) << 4),
                           static_cast<const uint16_t*>(job.q) + (there ? at + u * 8 : 0), there);
      }
    };
    auto landed_q = [&](const AttnTile& t) {
      if (job.q_tma) return;
      if (H == 2 && w == 1 && rows_all - t.row0 <= kTcHalf) return;
      asm volatile("cp.async.wait_all;\n" ::: "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full[w]);
    };
    // the next tile's rows on their way into the L2: queries, mask, the own positions' result
    auto prefetch_rows = [&](int hd, int en) {
      AttnTile t;
      t.b = job.phase == kShared ? 0 : job.by_tiles.div(en);
      t.row0 = (en - t.b * job.row_tiles) * kTcR;
      int b, node, g;
      if (!attn_row(job, t, t.row0 + w * kTcHalf + tid, b, node, g)) return;
      const uint16_t* q = static_cast<const uint16_t*>(job.q) + b * job.lq.batch_stride +
                          node * job.lq.node_stride + (hd * job.G + g) * job.lq.head_stride;
      for (int d = 0; d < job.D; d += 64) prefetch_l2(q + d);
      if (job.phase == kShared) {
        const float* own = job.own_o + ((int64_t)hd * job.B * job.by_ng.d + t.row0 +
                                        w * kTcHalf + tid) * DP;
#pragma unroll
        for (int d = 0; d < DP; d += 32) prefetch_l2(own + d);
      } else if (job.mask) {
        prefetch_l2(job.mask + ((int64_t)b * job.N + node) * job.N);
      }
    };
    // Page numbers of kTcCheck blocks, two boxes of each lane, read ahead (0 past the last
    // visible key: masked there).  Only where one is no page are the keys of the blocks looked
    // at one by one.
    auto page_at = [&](const AttnTile& t, int pos0, int box) {
      const int pos = pos0 + box * box_rows;
      if (box >= kTcCheck * boxes || pos >= t.kend) return 0;
      return job.table[(int64_t)t.b * job.max_pages + job.pd.div(pos)];  // kend lies within it
    };
    AttnTile t = attn_tile<kTcR, kTcKB>(job, walk.entry, lens);
    if (walk.left > 0) {
      load_q(walk.head, t);
      landed_q(t);
    }
    int ahead_a = page_at(t, t.kbeg + walk.unit * kTcKB, lane);
    int ahead_b = page_at(t, t.kbeg + walk.unit * kTcKB, lane + 32);
    int4 desc = make_int4(0, 0, 0, kSlotNone);
    while (walk.left > 0) {
      walk.take(t.blocks);
      const int head = walk.head, entry = walk.entry, block = walk.first, nb = walk.blocks;
      walk.next(job);
      const bool more = walk.left > 0;
      lens = attn_lens(job, walk.entry);
      const int halves = H == 2 && rows_all - t.row0 > kTcHalf ? 2 : 1;
      const int seg0 = t.kbeg + block * kTcKB;
      if (nb != t.blocks) {
        if (block == 0) {
          desc.x = 1;
          desc.y = head;
          desc.z = entry;
        } else {
          desc.w = block + nb == t.blocks ? kSlotEnd : kSlotMiddle;
        }
      }
      if (w < halves) {
        const int r = t.row0 + w * kTcHalf + tid;
        int rb, node, g;
        const bool real = attn_row(job, t, r, rb, node, g);
        float m = -CUDART_INF_F, l = 0.f;
        bool bad = false;
        for (int i = 0; i < nb; ++i) {
          const int pos0 = seg0 + i * kTcKB;
          if (i % kTcCheck == 0) {
            bad = __any_sync(kFull, (unsigned)ahead_a >= (unsigned)job.n_pages ||
                                        (unsigned)ahead_b >= (unsigned)job.n_pages);
            ahead_a = page_at(t, pos0 + kTcCheck * kTcKB, lane);
            ahead_b = page_at(t, pos0 + kTcCheck * kTcKB, lane + 32);
          }
          const bool drafts = pos0 + kTcKB > t.clear;  // rows may differ in what they see
          uint32_t sees[4];
          if (drafts || bad) {
            // bit k of word j: this row sees key 32 j + k of the block; at first those that every
            // row sees (without a mask the first drafts are among them)
            const int lim = t.clear - pos0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int n = min(max(lim - 32 * j, 0), 32);
              sees[j] = n == 32 ? kFull : (1u << n) - 1u;
            }
            if (drafts && job.phase == kOwn) {
              const int from = max(pos0, t.prefix), to = min(pos0 + kTcKB, t.kend);
              if (!job.mask) {
                const int end = min(to - t.prefix, node + 1) + (t.prefix - pos0);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const int n = min(max(end - 32 * j, 0), 32);
                  sees[j] = n == 32 ? kFull : (1u << n) - 1u;
                }
              } else {
                // the warp reads its nodes' mask rows together, 32 keys of a node at a time
                const int n0 = __shfl_sync(kFull, node, 0);
                const int n1 = min(__shfl_sync(kFull, node, 31), t.count - 1);
                const uint8_t* mrow = job.mask + ((int64_t)t.b * job.N + n0) * job.N - t.prefix;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const int p = pos0 + 32 * j + lane;
                  if (p - lane >= to || p - lane + 32 <= from) continue;
                  const bool in = p >= from && p < to;
                  for (int n = n0; n <= n1; n += 8) {
                    uint8_t x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                      x[e] = in && n + e <= n1 ? mrow[(int64_t)(n + e - n0) * job.N + p] : (uint8_t)0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                      const unsigned bits = __ballot_sync(kFull, x[e] != 0);
                      if (node == n + e) sees[j] |= bits;
                    }
                  }
                }
              }
            }
            if (bad) {
              const int mine = page_at(t, pos0, lane);
              const unsigned ok = __ballot_sync(
                  kFull, lane >= boxes || (unsigned)mine < (unsigned)job.n_pages);
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
          if (drafts || bad) {
            // keys the row does not see become -inf where they lie, in a small loop of its own:
            // the code that every block runs stays short (it does not fit the nearest
            // instruction caches as it is)
#pragma unroll 1
            for (int ch = 0; ch < kTcKB; ch += 16) {
              const uint32_t word = ch < 64 ? (ch < 32 ? sees[0] : sees[1])
                                            : (ch < 96 ? sees[2] : sees[3]);
              const uint32_t bits = word >> (ch & 16);
              uint32_t x[16];
              tc05_ld16(t_s + ch, x);
              tc05_wait_ld();
              tc05_landed16(x);
#pragma unroll
              for (int k = 0; k < 16; ++k)
                if (!((bits >> k) & 1u)) x[k] = 0xff800000u;
              tc05_st16(t_s + ch, x);
            }
            tc05_wait_st();
          }
          uint32_t s[kTcKB];
          tc05_ld32(t_s, s);
          tc05_ld32(t_s + 32, s + 32);
          tc05_ld32(t_s + 64, s + 64);
          tc05_ld32(t_s + 96, s + 96);
          tc05_wait_ld();
          tc05_landed(s);
          tc05_landed(s + 32);
          tc05_landed(s + 64);
          tc05_landed(s + 96);
          float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
          for (int k = 0; k < kTcKB; k += 8)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              mx[q] = fmaxf(mx[q], fmaxf(__uint_as_float(s[k + 2 * q]), __uint_as_float(s[k + 2 * q + 1])));
          const float mn = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), m);
          const bool rise = mn > m && (m == -CUDART_INF_F || (mn - m) * c > kTcLazy);
          if (__any_sync(kFull, rise)) {
            const float a = (rise && m != -CUDART_INF_F) ? ex2_approx((m - mn) * c)
                            : (rise ? 0.f : 1.f);
            if (i > 0) {  // (these scores were issued after the last product of the output)
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
          if (drafts) {
            // values past the last visible key leave the product, and so do infinities and
            // NaN among the drafts (a row that does not see them has weight 0 for them)
            const uint32_t ev = ent + 2 * i + 1;
            wait(&sh.full[ev % NST], (ev / NST) & 1u);
            constexpr int CPR = DP / 8;
            const int k0 = max(t.clear - pos0, 0), kn = min(t.kend - pos0, kTcKB);
            unsigned char* vb = base_p + Cfg::kQBytes + (ev % NST) * Cfg::kStageBytes;
            auto unit_at = [&](int x) {
              const int key = x / CPR, u = x % CPR;
              return reinterpret_cast<uint4*>(vb + (u >> 3) * Cfg::kChunkBytes + key * 128 +
                                              (((u & 7) ^ (key & 7)) << 4));
            };
            const int step = halves * kTcHalf;
#pragma unroll 1
            for (int x = k0 * CPR + w * kTcHalf + tid; x < kTcKB * CPR; x += step) {
              uint4* at = unit_at(x);
              const uint4 v = x < kn * CPR ? *at : make_uint4(~0u, ~0u, ~0u, ~0u);
              if (!unit_nonfinite<uint16_t>(v)) continue;
              uint32_t z[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                if ((z[q] & 0x7f800000u) == 0x7f800000u) z[q] &= 0xffffu;
                if ((z[q] & 0x7f80u) == 0x7f80u) z[q] &= 0xffff0000u;
              }
              *at = make_uint4(z[0], z[1], z[2], z[3]);
              if (x < kn * CPR) *((volatile int*)&sh.poison) = 1;
            }
            fence_proxy_async_smem();
            if (halves == 2) half_barrier<3, 2 * kTcHalf>();
            else half_barrier<2, kTcHalf>();
          }
          const float mc = m == -CUDART_INF_F ? 0.f : m * c;
          const float2 c2 = make_float2(c, c), n2 = make_float2(-mc, -mc);
          float2 sum = make_float2(0.f, 0.f), sum2 = sum;
          uint32_t* z = s + 64;
#pragma unroll
          for (int part = 1; part >= 0; --part) {
            if (part == 0) {
              tc05_ld32(t_s, z);
              tc05_ld32(t_s + 32, z + 32);
              tc05_wait_ld();
              tc05_landed(z);
              tc05_landed(z + 32);
            }
            uint32_t p[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              float2 x = fma_f32x2(make_float2(__uint_as_float(z[2 * k]),
                                               __uint_as_float(z[2 * k + 1])), c2, n2);
              x.x = ex2_approx(x.x);
              x.y = ex2_approx(x.y);
              if (k & 1) sum = add_f32x2(sum, x);
              else sum2 = add_f32x2(sum2, x);
              p[k] = pack_bf16(x.x, x.y);
            }
            tc05_st32(t_s + kTcP + 32 * part, p);
            tc05_wait_st();
            tc05_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full[w][part]);
          }
          if (i == 0 && more) prefetch_rows(walk.head, walk.entry);
          sum = add_f32x2(sum, sum2);
          l += sum.x + sum.y;
        }
        // the last scores are read: the half's queries may be replaced
        const AttnTile t_next = attn_tile<kTcR, kTcKB>(job, walk.entry, lens);
        if (more) load_q(walk.head, t_next);
        ahead_a = page_at(t_next, t_next.kbeg, lane);
        ahead_b = page_at(t_next, t_next.kbeg, lane + 32);

        // ---- epilogue.  Each thread scales its row; the rows leave through the warp's staging
        // area, so that a store fills whole sectors. ----
        const bool whole = nb == t.blocks;
        const bool leave = job.phase == kOwn && job.shared_len > 0;  // for the shared positions
        const bool wide = !whole || leave;                           // fp32 rows
        const int slot = 2 * cta + (block == 0 ? 1 : 0);
        const int rr = w * kTcHalf + tid;
        const int64_t own_row =
            ((int64_t)head * job.B + (job.phase == kShared ? 0 : rb)) * job.by_ng.d + r;
        const bool prior = whole && job.phase == kShared;
        int64_t to = -1;  // this row's destination
        if (!whole) to = ((int64_t)slot * kTcR + rr) * DP;
        else if (real) to = leave ? own_row * DP
                                  : rb * job.lo.batch_stride + node * job.lo.node_stride +
                                        (head * job.G + g) * job.lo.head_stride;
        // fp32 rows leave as 16 columns, four lanes to the 64 bytes of a row: this lane's part of
        // the rows lane / 4 + 8 i of the warp
        const int sub = lane & 3;
        int64_t src[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          src[i] = __shfl_sync(kFull, prior && real ? own_row * DP : (int64_t)-1,
                               (lane >> 2) + 8 * i);
        unsigned char* stage = base_p + Cfg::kQBytes + NST * Cfg::kStageBytes +
                               (w * 4 + (warp & 3)) * 32 * kTcStagePitch;
        unsigned char* stage_row = stage + lane * kTcStagePitch;
        unsigned char* stage_out = stage + (lane >> 2) * kTcStagePitch + sub * 16;
        float4 ahead[4], ahead2[4];  // the own positions' result, 16 and 32 columns ahead
        auto fetch = [&](int col) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            ahead2[i] = src[i] >= 0 && col < DP
                            ? *reinterpret_cast<const float4*>(job.own_o + src[i] + col + sub * 4)
                            : make_float4(0.f, 0.f, 0.f, 0.f);
        };
        if (prior) {
          fetch(0);
#pragma unroll
          for (int i = 0; i < 4; ++i) ahead[i] = ahead2[i];
          fetch(16);
        }
        const bool query = real && (!whole || leave || attn_query(job, rb, node));
        const float own_lse = prior && query ? job.own_lse[own_row] : -CUDART_INF_F;
        wait(&sh.o_full[w], seg & 1u);
        ++seg;
        if (more) landed_q(t_next);
        __syncwarp();
        tc05_fence_after();
        if (*((volatile int*)&sh.abort)) l = __int_as_float(0x7fc00000);
        if (*((volatile int*)&sh.poison) && job.phase == kOwn) {
          const int seg1 = min(seg0 + nb * kTcKB, t.kend);
#pragma unroll 1
          for (int ch = 0; ch < DP; ch += 16) {
            uint32_t o[16];
            __syncwarp();
            tc05_ld16(t_o + ch, o);
            tc05_wait_ld();
            tc05_landed16(o);
            float x[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) x[k] = __uint_as_float(o[k]);
            if (real)
              add_nonfinite<uint16_t, 16>(job, t, head, node, max(t.clear, seg0), seg1, ch, x);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(x[k]);
            __syncwarp();
            tc05_st16(t_o + ch, o);
          }
          tc05_wait_st();
        }
        const float m2 = m == -CUDART_INF_F ? m : m * c;
        // the row's weight, and the own positions' where they are joined
        bool some = true;
        float wo = 1.f, w_own = 0.f;
        if (!whole) {
          job.part_ms[(slot * 2) * kTcR + rr] = m2;
          job.part_ms[(slot * 2 + 1) * kTcR + rr] = l;
        } else {
          const AttnJoin j = attn_join(m2, l, own_lse);
          some = query && l != 0.f;
          wo = j.w;
          w_own = query ? j.w_own : 0.f;
          if (leave && real) {
            job.own_lse[own_row] = j.lse2;
          } else if (real && job.lse) {
            job.lse[((int64_t)rb * job.N + node) * job.Hq + head * job.G + g] =
                query ? j.lse2 * 0.693147180559945309f : -CUDART_INF_F;
          }
        }
#pragma unroll 1
        for (int ch = 0; ch < DP; ch += 16) {
          uint32_t o[16];
          __syncwarp();
          tc05_ld16(t_o + ch, o);
          tc05_wait_ld();
          tc05_landed16(o);
          float of[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) of[k] = some ? __uint_as_float(o[k]) * wo : 0.f;
          if (prior) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              *reinterpret_cast<float4*>(stage_out + 8 * i * kTcStagePitch) = ahead[i];
              ahead[i] = ahead2[i];
            }
            fetch(ch + 32);
            __syncwarp();
            const bool joined = w_own != 0.f;
#pragma unroll
            for (int k = 0; k < 16; k += 4) {
              const float4 x = *reinterpret_cast<const float4*>(stage_row + k * 4);
              of[k] += joined ? x.x * w_own : 0.f;
              of[k + 1] += joined ? x.y * w_own : 0.f;
              of[k + 2] += joined ? x.z * w_own : 0.f;
              of[k + 3] += joined ? x.w * w_own : 0.f;
            }
            __syncwarp();
          }
          if (wide) {
            float* out = whole ? job.own_o : job.part_o;
#pragma unroll
            for (int k = 0; k < 16; k += 4)
              *reinterpret_cast<float4*>(stage_row + k * 4) =
                  make_float4(of[k], of[k + 1], of[k + 2], of[k + 3]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int64_t dst = __shfl_sync(kFull, to, (lane >> 2) + 8 * i);
              if (dst >= 0)
                *reinterpret_cast<float4*>(out + dst + ch + sub * 4) =
                    *reinterpret_cast<const float4*>(stage_out + 8 * i * kTcStagePitch);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 16; k += 8)
              *reinterpret_cast<uint4*>(stage_row + k * 2) =
                  make_uint4(pack_bf16(of[k], of[k + 1]), pack_bf16(of[k + 2], of[k + 3]),
                             pack_bf16(of[k + 4], of[k + 5]), pack_bf16(of[k + 6], of[k + 7]));
            __syncwarp();
            const int unit = lane & 1;  // two lanes to the 32 bytes of a row
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int row = (lane >> 1) + 16 * i;
              const int64_t dst = __shfl_sync(kFull, to, row);
              if (dst >= 0 && ch + unit * 8 < job.D)
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(job.out) + dst + ch + unit * 8) =
                    *reinterpret_cast<const uint4*>(stage + row * kTcStagePitch + unit * 16);
            }
          }
        }
        tc05_fence_before();
        t = t_next;
      } else {
        t = attn_tile<kTcR, kTcKB>(job, walk.entry, lens);  // this half idles in this tile
        ahead_a = page_at(t, t.kbeg, lane);
        ahead_b = page_at(t, t.kbeg, lane + 32);
        if (more) {
          load_q(walk.head, t);
          landed_q(t);
        }
      }
      ent += 2 * nb;
    }
    if (threadIdx.x == 64) job.part_desc[cta] = desc;
  }
  tc05_fence_before();
  __syncthreads();
  tc05_fence_after();
  if (warp == 1) tc05_dealloc(tmem, Cfg::kTmemCols);
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

// The queries as [batch][node][head][d], a box being the rows of a half: 64 d of a key head's
// query heads in 128 / G nodes.  The shared positions' tiles run over the nodes of all
// sequences, so there batches and nodes have to be one direction.
bool make_query_map(CUtensorMap* map, const AttnJob& job) {
  EncodeTiledFn fn = encode_fn();
  if (!fn || kTcHalf % job.G != 0) return false;
  int64_t nodes = job.N, batches = job.B, step = job.lq.node_stride;
  if (job.phase == kShared) {
    if (job.N == 1) step = job.lq.batch_stride;
    else if (job.B > 1 && job.lq.batch_stride != job.N * job.lq.node_stride) return false;
    nodes *= batches;
    batches = 1;
  }
  const cuuint64_t dims[4] = {(cuuint64_t)job.D, (cuuint64_t)job.Hq, (cuuint64_t)nodes,
                              (cuuint64_t)batches};
  const cuuint64_t strides[3] = {(cuuint64_t)job.lq.head_stride * 2, (cuuint64_t)step * 2,
                                 (cuuint64_t)job.lq.batch_stride * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)job.G, (cuuint32_t)(kTcHalf / job.G), 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(job.q), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DP, int H>
cudaError_t launch_tc(AttnJob job, int rows, cudaStream_t s, bool* taken) {
  using Cfg = TcCfg<DP, H>;
  const int box = tc_box_rows(job.pd.size);
  CUtensorMap tm_k, tm_v, tm_q;
  *taken = make_cache_map(&tm_k, job.k, job, box) && make_cache_map(&tm_v, job.v, job, box);
  if (!*taken) return cudaSuccess;
  job.q_tma = make_query_map(&tm_q, job);
  if (!job.q_tma) tm_q = tm_k;  // not used
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    e = cudaFuncSetAttribute(attn_tc_kernel<DP, H>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Cfg::kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev] = true;
  }
  job.row_tiles = (rows + Cfg::kR - 1) / Cfg::kR;
  job.entries = job.phase == kShared ? job.row_tiles : job.row_tiles * job.B;
  job.by_tiles = FastDiv::make(job.row_tiles);
  const int most = kAttnTcSlots / Cfg::kR, sms = device_sm_count() * (3 - H);
  const int grid = sms < most ? sms : most;
  attn_tc_kernel<DP, H><<<grid, Cfg::kThreads, Cfg::kSmem, s>>>(tm_k, tm_v, tm_q, job, box);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_attn_combine(job, DP, Cfg::kR, grid, s);
}

int64_t tc_rows(const AttnJob& job) {
  return job.phase == kShared ? (int64_t)job.B * job.N * job.G : (int64_t)job.N * job.G;
}

}  // namespace

// Few rows do not pay for 128-row products (16 rows a key head on 64 x 2000 positions: 115 us in
// the few-rows kernel; 20 rows: 121 here, 208 there), a box of fewer than 8 rows does not fill a swizzle
// group, and the maximum is taken, and masked keys set to -inf, before the scaling.
bool attn_tc_fits(const AttnJob& job, spec_dtype dtype) {
  return dtype == SPEC_BF16 && job.scale_log2 > 0.f && job.pd.size % 8 == 0 && job.n_pages > 0 &&
         tc_rows(job) > kAttnRowsTile;
}

cudaError_t launch_attn_tc(const AttnJob& job, cudaStream_t s, bool* taken) {
  const int rows = (int)tc_rows(job);
  if (rows <= kTcHalf)
    return job.D <= 64 ? launch_tc<64, 1>(job, rows, s, taken) : launch_tc<128, 1>(job, rows, s, taken);
  return job.D <= 64 ? launch_tc<64, 2>(job, rows, s, taken) : launch_tc<128, 2>(job, rows, s, taken);
}

}  // namespace svk
