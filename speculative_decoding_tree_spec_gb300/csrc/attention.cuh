// attention.cuh -- the work list of the paged tree attention, shared by its kernels.
//
// Rows: the query heads that read one key head are taken together, row r = node * G + g of
// sequence b (G = query heads per key head), in tiles of R rows.  A tile's keys are cut into
// blocks of KB positions; a tile is max(1, blocks) + C units of work, C standing for its fixed
// costs (queries, epilogue), numbered key head by key head and tile by tile.  CTA j of n takes
// the units [U j / n, U (j + 1) / n): every CTA does the same amount of work however the
// lengths differ.  A tile that lies in one CTA is finished there; of a tile cut between CTAs each CTA leaves its part (running maximum, sum,
// unnormalised output) in one of its two slots and attn_combine_kernel joins the parts in
// the order of the keys.  The split depends on the lengths and the grid alone, so a call is
// reproducible bit for bit.
//
// Two phases: kOwn takes each sequence's own positions (from shared_len on); kShared, after it,
// the positions all sequences share, for the rows of all sequences at once (row r = (b * N +
// node) * G + g).  With shared positions kOwn leaves a normalised fp32 result that kShared
// joins with its own: the shared tiles are the long ones, beside which the join costs least
// (in the first measurement of both orders the join in the short own tiles made the own part of
// 256 x 26-node trees on 16 to 400 positions 212 us instead of 163, and the shared part 45 us
// shorter; the own part takes 140 us now, 131 and its join of cut tiles).
#pragma once

#include <cuda_bf16.h>

#include "paged.cuh"

namespace svk {

constexpr int kAttnMaxCtas = 512;   // grid limit: two slots per CTA in the workspace
constexpr int kAttnTcSlots = 256 * 256;  // tensor-memory kernel: limit of CTAs * rows of a tile
constexpr int kAttnTcKeys = 128;  // keys of the tensor-memory kernel's block
constexpr int kAttnRowsTile = 16;  // rows of the few-rows kernel's tile

enum AttnPhase { kOwn = 0, kShared = 1 };

struct AttnJob {
  const void *q, *k, *v;
  void* out;
  float* lse;
  spec_node_layout lq, lo;                       // elements
  int64_t page_stride, pos_stride, head_stride;  // elements
  const int32_t *table, *prefix, *counts;
  const uint8_t* mask;
  int B, N, Hq, Hkv, G, D, n_pages, max_pages, shared_len;
  int row_tiles;   // tiles per sequence (kOwn) or in all (kShared)
  int entries;     // tiles of one key head
  PageDiv pd;
  FastDiv by_g, by_ng, by_tiles;  // G, N * G, row_tiles
  float scale_log2;  // scale * log2(e)
  int phase;
  int q_tma;  // queries come by tensor map
  // result of the own positions where there are shared ones, [Hkv][B * N * G] rows:
  // normalised output (row pitch DP) and its log2-sum-exp2
  float* own_o;
  float* own_lse;
  // two slots per CTA: [slot][R] maximum and sum, [slot][R][DP] output
  float* part_ms;
  float* part_o;
  int4* part_desc;  // per CTA: {a tile is left open, key head, tile, what slot 0 holds}
};

bool attn_tc_fits(const AttnJob& job, spec_dtype dtype);
// The tensor-memory kernel and its join; *taken = false where the cache's strides make no
// tensor map (nothing was launched).
cudaError_t launch_attn_tc(const AttnJob& job, cudaStream_t s, bool* taken);
cudaError_t launch_attn_combine(const AttnJob& job, int DP, int R, int ctas, cudaStream_t s);

// What slot 0 of a CTA holds: nothing, the middle of a tile, the end of one.
enum { kSlotNone = 0, kSlotMiddle = 1, kSlotEnd = 2 };

// One tile's rows and keys.
struct AttnTile {
  int b;            // sequence (0 for the shared positions)
  int row0;         // first row
  int prefix, count;
  int kbeg, kend;   // positions its rows can see at most
  int clear;        // positions below it are seen by every query of the tile
  int blocks;       // units
};

// The lengths a tile needs from memory, read ahead of its use.
struct AttnLens {
  int prefix, count;
};
__device__ __forceinline__ AttnLens attn_lens(const AttnJob& job, int entry) {
  AttnLens x{0, 0};
  if (job.phase == kOwn && entry < job.entries) {
    const int b = job.by_tiles.div(entry);
    x.prefix = job.prefix[b];
    x.count = job.counts ? job.counts[b] : job.N;
  }
  return x;
}

template <int R, int KB>
__device__ __forceinline__ AttnTile attn_tile(const AttnJob& job, int entry, const AttnLens& lens) {
  AttnTile t;
  const int cap = job.max_pages * job.pd.size;
  if (job.phase == kShared) {
    t.b = 0;
    t.row0 = entry * R;
    t.prefix = job.shared_len;
    t.count = job.N;
    t.kbeg = 0;
    t.kend = t.clear = min(job.shared_len, cap);
  } else {
    t.b = job.by_tiles.div(entry);
    t.row0 = (entry - t.b * job.row_tiles) * R;
    t.prefix = min(max(lens.prefix, 0), cap);  // no position beyond the table exists
    t.count = min(max(lens.count, 0), job.N);
    if (t.prefix < job.shared_len) t.count = 0;  // not a sequence behind the shared prefix
    t.kbeg = job.shared_len;
    const int first = job.by_g.div(t.row0);
    const int last = job.by_g.div(min(t.row0 + R, job.N * job.G) - 1);
    int64_t end = (int64_t)t.prefix + (job.mask ? t.count : min(t.count, last + 1));
    if (first >= t.count) end = t.kbeg;  // only padding rows
    t.kend = (int)max((int64_t)t.kbeg, min(end, (int64_t)cap));
    t.clear = min(t.kend, t.prefix);
    if (!job.mask && first < t.count)
      t.clear = (int)min((int64_t)t.kend, (int64_t)t.prefix + first + 1);
  }
  t.blocks = max(1, (t.kend - t.kbeg + KB - 1) / KB);
  return t;
}
template <int R, int KB>
__device__ __forceinline__ AttnTile attn_tile(const AttnJob& job, int entry) {
  return attn_tile<R, KB>(job, entry, attn_lens(job, entry));
}

// This CTA's units and where the first one lies: key head, tile, unit in it.
struct AttnRange {
  int64_t units;
  int head, entry, unit;
};

// A walk over the units of a CTA, tile by tile.  The blocks of a tile are its first units.
template <int C>
struct AttnWalk {
  int64_t left;
  int head, entry, unit;  // the next tile to take, and the unit to start at
  int first, blocks;      // taken: first block and number of blocks

  __device__ __forceinline__ explicit AttnWalk(const AttnRange& r)
      : left(r.units), head(r.head), entry(r.entry), unit(r.unit), first(0), blocks(0) {}
  // Takes the units of a tile of `tile_blocks` blocks.
  __device__ __forceinline__ void take(int tile_blocks) {
    const int n = (int)min((int64_t)(tile_blocks + C - unit), left);
    first = min(unit, tile_blocks);
    blocks = min(unit + n, tile_blocks) - first;
    left -= n;
  }
  __device__ __forceinline__ int next_entry(const AttnJob& job) const {
    return entry + 1 == job.entries ? 0 : entry + 1;
  }
  __device__ __forceinline__ void next(const AttnJob& job) {
    unit = 0;
    if (++entry == job.entries) {
      entry = 0;
      ++head;
    }
  }
};

// All NT threads of the block call this.  Thread i sums the units of a run of tiles; a scan
// over the threads gives a key head's units and the run that holds the first one.
template <int R, int KB, int C, int NT>
__device__ __forceinline__ AttnRange attn_range(const AttnJob& job, int cta, int ctas) {
  __shared__ int64_t warp_sum[NT / 32];
  __shared__ int found[3];
  const int run = (job.entries + NT - 1) / NT;
  const int e0 = (int)threadIdx.x * run, e1 = min(e0 + run, job.entries);
  int64_t mine = 0;
  for (int e = e0; e < e1; ++e) mine += attn_tile<R, KB>(job, e).blocks + C;
  int64_t inc = mine;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(kFull, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int64_t before = 0, per_head = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    per_head += warp_sum[w];
  }
  const int64_t total = per_head * job.Hkv;
  const int64_t u0 = total * cta / ctas, u1 = total * (cta + 1) / ctas;
  AttnRange r;
  r.units = u1 - u0;
  r.head = (int)(u0 / per_head);
  int64_t rest = u0 - r.head * per_head - (before + inc - mine);
  if (rest >= 0 && rest < mine) {
    int e = e0, n;
    for (;; ++e) {
      n = attn_tile<R, KB>(job, e).blocks + C;
      if (rest < n) break;
      rest -= n;
    }
    // a CTA that would start behind the tile's blocks starts with the next tile
    const bool behind = rest >= n - C;
    found[0] = behind ? e + 1 : e;
    found[1] = behind ? 0 : (int)rest;
    found[2] = behind ? (int)(n - rest) : 0;
  }
  __syncthreads();
  r.entry = found[0];
  r.unit = found[1];
  if (r.units > 0) r.units -= min((int64_t)found[2], r.units);
  if (r.entry == job.entries) {
    r.entry = 0;
    ++r.head;
  }
  return r;
}

// Whether row r of the tile is a query (not padding), and its node.
__device__ __forceinline__ bool attn_row(const AttnJob& job, const AttnTile& t, int r, int& b,
                                         int& node, int& g) {
  if (job.phase == kShared) {
    b = job.by_ng.div(r);
    r -= b * job.by_ng.d;
  } else {
    b = t.b;
  }
  node = job.by_g.div(r);
  g = r - node * job.G;
  return job.phase == kShared ? b < job.B : node < job.N;
}

// Whether node n of the tile's sequence sees position t >= prefix (t below kend).
__device__ __forceinline__ bool attn_sees_draft(const AttnJob& job, const AttnTile& t, int n,
                                                int pos) {
  const int j = pos - t.prefix;
  if (j >= t.count || n >= t.count) return false;
  return job.mask ? job.mask[((int64_t)t.b * job.N + n) * job.N + j] != 0 : j <= n;
}

__device__ __forceinline__ void cp_async16_or_zero(uint32_t smem, const void* gmem, bool real) {
  const int n = real ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem), "l"(gmem), "r"(n)
               : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T> __device__ __forceinline__ T from_float(float x);
template <> __device__ __forceinline__ float from_float<float>(float x) { return x; }
template <> __device__ __forceinline__ uint16_t from_float<uint16_t>(float x) {
  return __bfloat16_as_ushort(__float2bfloat16(x));
}

// Whether a 16-byte unit holds an infinity or a NaN.
template <typename T> __device__ __forceinline__ bool unit_nonfinite(const uint4& x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (sizeof(T) == 4) {
      bad |= (w[i] & 0x7f800000u) == 0x7f800000u;
    } else {
      bad |= (w[i] & 0x7f800000u) == 0x7f800000u || (w[i] & 0x7f80u) == 0x7f80u;
    }
  }
  return bad;
}

// Whether the result of row (b, node) counts: a query that is no padding, of a sequence that
// does stand behind the shared positions.
__device__ __forceinline__ bool attn_query(const AttnJob& job, int b, int node) {
  if (job.counts && node >= job.counts[b]) return false;
  return job.shared_len == 0 || job.prefix[b] >= job.shared_len;
}

// Weights of a row's result (m, l, log2 units) and of the own positions' result left for it
// (its log2-sum-exp2): out = o * w + own * w_own, and their log2-sum-exp2.
struct AttnJoin {
  float w, w_own, lse2;
};
__device__ __forceinline__ AttnJoin attn_join(float m, float l, float own) {
  AttnJoin j;
  j.w = l == 0.f ? 0.f : 1.f / l;
  j.w_own = 0.f;
  j.lse2 = l == 0.f ? -CUDART_INF_F : m + log2f(l);
  if (own != -CUDART_INF_F) {
    const float top = fmaxf(own, j.lse2);
    const float eo = exp2f(own - top), es = l == 0.f ? 0.f : exp2f(j.lse2 - top);
    j.w_own = eo / (eo + es);
    j.w = l == 0.f ? 0.f : es / (eo + es) / l;
    j.lse2 = top + log2f(eo + es);
  }
  return j;
}

// One row's result: its part (m, l, o[0..n) of columns c0..), left for the shared positions or
// joined with what the own positions left, and written.
template <typename T, int C>
__device__ __forceinline__ void write_row(const AttnJob& job, const AttnTile& t, int head, int r,
                                          int c0, int DP, float m, float l, float (&o)[C]) {
  int b, node, g;
  if (!attn_row(job, t, r, b, node, g)) return;
  const int64_t row = ((int64_t)head * job.B + (job.phase == kShared ? 0 : b)) * job.by_ng.d + r;
  const bool leave = job.phase == kOwn && job.shared_len > 0;
  const bool query = leave || attn_query(job, b, node);
  const AttnJoin j = attn_join(m, l, job.phase == kShared && query ? job.own_lse[row] : -CUDART_INF_F);
  const bool some = query && l != 0.f;
#pragma unroll
  for (int i = 0; i < C; ++i) o[i] = some ? o[i] * j.w : 0.f;
  if (query && j.w_own != 0.f) {
    const float* own = job.own_o + row * DP + c0;
#pragma unroll
    for (int i = 0; i < C; i += 4) {
      const float4 x = *reinterpret_cast<const float4*>(own + i);
      o[i] += x.x * j.w_own;
      o[i + 1] += x.y * j.w_own;
      o[i + 2] += x.z * j.w_own;
      o[i + 3] += x.w * j.w_own;
    }
  }
  if (leave) {
    float4* dst = reinterpret_cast<float4*>(job.own_o + row * DP + c0);
#pragma unroll
    for (int i = 0; i < C; i += 4) dst[i / 4] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
    if (c0 == 0) job.own_lse[row] = j.lse2;
    return;
  }
  const int h = head * job.G + g;
  T* dst = static_cast<T*>(job.out) + b * job.lo.batch_stride + node * job.lo.node_stride +
           h * job.lo.head_stride;
  constexpr int E = 16 / (int)sizeof(T);
#pragma unroll
  for (int i = 0; i < C; i += E) {
    if (c0 + i < job.D) {
      T x[E];
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = from_float<T>(o[i + e]);
      *reinterpret_cast<uint4*>(dst + c0 + i) = *reinterpret_cast<const uint4*>(x);
    }
  }
  if (c0 == 0 && job.lse)
    job.lse[((int64_t)b * job.N + node) * job.Hq + h] =
        query ? j.lse2 * 0.693147180559945309f : -CUDART_INF_F;
}

// Infinities and NaN among the draft positions' values [from, to) that row (node) sees.  A
// tile in which some rows do not see a key multiplies it by 0 for them, so such values are
// taken out of the product (as 0) and added here for the rows that do see them.
template <typename T, int C>
static __device__ __noinline__ void add_nonfinite(const AttnJob& job, const AttnTile& t,
                                                  int head, int node, int from, int to, int c0,
                                                  float* o) {
  const int32_t* row = job.table + (int64_t)t.b * job.max_pages;
  for (int pos = from; pos < to; ++pos) {
    if (!attn_sees_draft(job, t, node, pos)) continue;
    const int64_t off = paged_offset(row, job.max_pages, job.n_pages, job.pd, job.page_stride,
                                     job.pos_stride, pos);
    if (off < 0) continue;
    const T* v = static_cast<const T*>(job.v) + off + head * job.head_stride;
    for (int i = 0; i < C && c0 + i < job.D; ++i) {
      const float x = Elt<T>::at(v, c0 + i);
      if (!(fabsf(x) < CUDART_INF_F)) o[i] += x;
    }
  }
}

}  // namespace svk
