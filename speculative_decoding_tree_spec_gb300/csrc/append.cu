// append.cu -- keys and values of new tokens into a paged cache, the keys' rotary position
// rotation applied on the way, and the tokens' queries rotated with them.  This is the step
// before the target model's pass over a draft tree: node n of tree b is stored at position
// prefix_len[b] + n and rotated by prefix_len[b] + position_ids[b][n], its depth in the tree
// (the position ids spec_tree_build gives), so that a later commit can move an accepted node
// to position prefix_len[b] + depth without rotating it again.
//
//   x'[i]     = x[i] cos_r[i] - x[i + h] sin_r[i]
//   x'[i + h] = x[i + h] cos_r[i] + x[i] sin_r[i],  i < h = rot / 2
// (interleaved: the pairs are (2 i, 2 i + 1)); elements from rot on pass through.  fp32
// arithmetic, one rounding to the cache's type.
#include <cuda_bf16.h>

#include "paged.cuh"

namespace svk {

namespace {

constexpr int kAppendThreads = 128;
constexpr int kAppendBatch = 3;  // heads whose loads a thread has in flight

struct AppendJob {
  const unsigned char *q, *k, *v;
  unsigned char *out_q, *kc, *vc;
  spec_node_layout lq, lo, lk, lv;               // bytes
  int64_t page_stride, pos_stride, head_stride;  // bytes
  const int32_t *table, *prefix, *counts, *ids;
  const float* cos_sin;
  int N, Hq, Hkv, max_pages, n_pages, n_positions, rot, vecs;
  PageDiv pd;
};

template <typename T>
__device__ __forceinline__ uint4 pack_unit(const float (&f)[Elt<T>::kPerUnit]);
template <>
__device__ __forceinline__ uint4 pack_unit<float>(const float (&f)[4]) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                    __float_as_uint(f[3]));
}
template <>
__device__ __forceinline__ uint4 pack_unit<uint16_t>(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// What bounds it: the tokens' bytes, each read and written once; 64 trees of 60 nodes with 32
// query and 8 key heads of 128 in bf16 (96 MB) take 15.7 us, 90 % of the measured copy bandwidth.
// One token takes 4.2 us, the chain prefix -> cosines and page table -> rows -> stores.
//
// One block per token.  A thread owns one pair of 16-byte units of a head (the two halves
// of a rotated pair where the pairs are split) and walks the heads, so it reads its cosines
// and sines once.
template <typename T, bool INTER>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(AppendJob job) {
  constexpr int E = Elt<T>::kPerUnit;
  const int b = (int)(blockIdx.x / job.N), n = (int)(blockIdx.x % job.N);
  const int pre = max(job.prefix[b], 0);
  const int count = job.counts ? min(job.counts[b], job.N) : job.N;
  int64_t r = pre;
  if (job.rot) r += job.ids ? job.ids[(int64_t)b * job.N + n] : n;
  const bool real = n < count && r >= 0 && (job.rot == 0 || r < job.n_positions);
  const int pairs = (job.vecs + 1) / 2;        // unit pairs of a head
  const int u = threadIdx.x % pairs, lane_head = threadIdx.x / pairs;
  const int heads_step = kAppendThreads / pairs;
  if (lane_head >= heads_step) return;
  const int rot_pairs = job.rot / (2 * E);     // unit pairs that are rotated
  const bool turn = u < rot_pairs;
  int ua, ub;                                  // this thread's units of a head
  if (INTER || !turn) {
    ua = 2 * u;
    ub = 2 * u + 1;
  } else {
    ua = u;
    ub = u + rot_pairs;
  }
  const bool has_b = ub < job.vecs;
  float cs[E], sn[E];
  if (real && turn) {
    const float* row = job.cos_sin + r * job.rot + (int64_t)u * E;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      cs[i] = row[i];
      sn[i] = row[job.rot / 2 + i];
    }
  }
  const int64_t t = (int64_t)pre + n;
  const int64_t slot = (real && t <= SPEC_MAX_POSITIONS)
      ? paged_offset(job.table + (int64_t)b * job.max_pages, job.max_pages, job.n_pages, job.pd,
                     job.page_stride, job.pos_stride, (int)t)
      : (int64_t)-1;
  auto rotate = [&](uint4& xa, uint4& xb) {
    float a[E], c[E];
    Elt<T>::unpack(xa, a);
    Elt<T>::unpack(xb, c);
    if (INTER) {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        const float x = a[2 * i], y = a[2 * i + 1];
        a[2 * i] = x * cs[i] - y * sn[i];
        a[2 * i + 1] = y * cs[i] + x * sn[i];
        const float z = c[2 * i], w = c[2 * i + 1];
        c[2 * i] = z * cs[E / 2 + i] - w * sn[E / 2 + i];
        c[2 * i + 1] = w * cs[E / 2 + i] + z * sn[E / 2 + i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float x = a[i], y = c[i];
        a[i] = x * cs[i] - y * sn[i];
        c[i] = y * cs[i] + x * sn[i];
      }
    }
    xa = pack_unit<T>(a);
    xb = pack_unit<T>(c);
  };
  // Heads in batches: the loads of a batch stand before its first store.
  const int total = job.Hq + 2 * job.Hkv;
  for (int h0 = lane_head; h0 < total; h0 += kAppendBatch * heads_step) {
    uint4 xa[kAppendBatch], xb[kAppendBatch];
    unsigned char* dst[kAppendBatch];
#pragma unroll
    for (int i = 0; i < kAppendBatch; ++i) {
      const int h = h0 + i * heads_step;
      dst[i] = nullptr;
      xa[i] = xb[i] = make_uint4(0, 0, 0, 0);
      if (h >= total) continue;
      const unsigned char* src;
      if (h < job.Hq) {
        src = job.q + b * job.lq.batch_stride + n * job.lq.node_stride + h * job.lq.head_stride;
        dst[i] = job.out_q + b * job.lo.batch_stride + n * job.lo.node_stride +
                 h * job.lo.head_stride;
      } else {
        const bool is_v = h >= job.Hq + job.Hkv;
        const int g = h - job.Hq - (is_v ? job.Hkv : 0);
        const spec_node_layout& l = is_v ? job.lv : job.lk;
        src = (is_v ? job.v : job.k) + b * l.batch_stride + n * l.node_stride + g * l.head_stride;
        if (slot >= 0) dst[i] = (is_v ? job.vc : job.kc) + slot + g * job.head_stride;
      }
      if (real && dst[i]) {
        xa[i] = *reinterpret_cast<const uint4*>(src + ua * 16);
        if (has_b) xb[i] = *reinterpret_cast<const uint4*>(src + ub * 16);
      }
    }
#pragma unroll
    for (int i = 0; i < kAppendBatch; ++i) {
      if (!dst[i]) continue;
      if (real && turn && h0 + i * heads_step < job.Hq + job.Hkv) rotate(xa[i], xb[i]);
      *reinterpret_cast<uint4*>(dst[i] + ua * 16) = xa[i];
      if (has_b) *reinterpret_cast<uint4*>(dst[i] + ub * 16) = xb[i];
    }
  }
}

bool misaligned(const spec_node_layout& l) {
  return ((l.batch_stride | l.node_stride | l.head_stride) & 15) != 0;
}

spec_node_layout in_bytes(const spec_node_layout& l, int64_t es) {
  return {l.batch_stride * es, l.node_stride * es, l.head_stride * es};
}

}  // namespace

int check_paged_layout(const spec_paged_layout& l, int32_t max_pages) {
  if (l.n_pages < 0 || l.page_size < 1 || l.n_kv_heads < 1 || l.head_dim < 1 || max_pages < 0 ||
      l.page_stride < 0 || l.pos_stride < 0 || l.head_stride < 0)
    return SPEC_ERR_INVALID_ARG;
  if ((int64_t)max_pages * l.page_size > SPEC_MAX_POSITIONS) return SPEC_ERR_TOO_LARGE;
  return SPEC_OK;
}

}  // namespace svk

using namespace svk;

extern "C" int spec_paged_append_rope(
    const void* q, spec_node_layout q_layout, void* out_q, spec_node_layout out_q_layout,
    const void* k, spec_node_layout k_layout, const void* v, spec_node_layout v_layout,
    spec_dtype dtype, int32_t B, int32_t N, int32_t n_q_heads, void* k_cache, void* v_cache,
    spec_paged_layout cache, const int32_t* page_table, int32_t max_pages,
    const int32_t* prefix_len, const int32_t* counts, const int32_t* position_ids,
    const float* cos_sin, int32_t n_positions, int32_t rot_dim, uint32_t flags,
    spec_stream_t stream) {
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_UNSUPPORTED_DTYPE;
  int rc = check_paged_layout(cache, max_pages);
  if (rc != SPEC_OK) return rc;
  if (B < 0 || N < 0 || n_q_heads < 0 || rot_dim < 0 || rot_dim > cache.head_dim ||
      n_positions < 0 || (flags & ~SPEC_ROPE_INTERLEAVED))
    return SPEC_ERR_INVALID_ARG;
  if (B == 0 || N == 0) return SPEC_OK;
  if (!k || !v || !k_cache || !v_cache || !page_table || !prefix_len ||
      (n_q_heads > 0 && (!q || !out_q)) || (rot_dim > 0 && !cos_sin))
    return SPEC_ERR_INVALID_ARG;
  if (cache.head_dim > SPEC_APPEND_MAX_HEAD_DIM) return SPEC_ERR_TOO_LARGE;
  const int64_t es = dtype == SPEC_F32 ? 4 : 2;
  const int unit = (int)(16 / es);
  if (cache.head_dim % unit != 0 || rot_dim % (2 * unit) != 0) return SPEC_ERR_MISALIGNED;
  AppendJob job{};
  job.lq = in_bytes(q_layout, es);
  job.lo = in_bytes(out_q_layout, es);
  job.lk = in_bytes(k_layout, es);
  job.lv = in_bytes(v_layout, es);
  job.page_stride = cache.page_stride * es;
  job.pos_stride = cache.pos_stride * es;
  job.head_stride = cache.head_stride * es;
  const uintptr_t bases = reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
                          reinterpret_cast<uintptr_t>(k_cache) |
                          reinterpret_cast<uintptr_t>(v_cache) |
                          (n_q_heads > 0 ? reinterpret_cast<uintptr_t>(q) |
                                               reinterpret_cast<uintptr_t>(out_q) : 0);
  if ((bases & 15u) || misaligned(job.lk) || misaligned(job.lv) ||
      (n_q_heads > 0 && (misaligned(job.lq) || misaligned(job.lo))) ||
      ((job.page_stride | job.pos_stride | job.head_stride) & 15))
    return SPEC_ERR_MISALIGNED;
  const int64_t tokens = (int64_t)B * N;
  if (tokens > 0x7fffffff) return SPEC_ERR_TOO_LARGE;
  job.q = static_cast<const unsigned char*>(q);
  job.k = static_cast<const unsigned char*>(k);
  job.v = static_cast<const unsigned char*>(v);
  job.out_q = static_cast<unsigned char*>(out_q);
  job.kc = static_cast<unsigned char*>(k_cache);
  job.vc = static_cast<unsigned char*>(v_cache);
  job.table = page_table;
  job.prefix = prefix_len;
  job.counts = counts;
  job.ids = position_ids;
  job.cos_sin = cos_sin;
  job.N = N;
  job.Hq = n_q_heads;
  job.Hkv = cache.n_kv_heads;
  job.max_pages = max_pages;
  job.n_pages = cache.n_pages;
  job.n_positions = n_positions;
  job.rot = rot_dim;
  job.vecs = cache.head_dim / unit;
  job.pd = PageDiv::make(cache.page_size);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool inter = flags & SPEC_ROPE_INTERLEAVED;
  const unsigned grid = (unsigned)tokens;
  if (dtype == SPEC_BF16) {
    if (inter) append_kernel<uint16_t, true><<<grid, kAppendThreads, 0, s>>>(job);
    else append_kernel<uint16_t, false><<<grid, kAppendThreads, 0, s>>>(job);
  } else {
    if (inter) append_kernel<float, true><<<grid, kAppendThreads, 0, s>>>(job);
    else append_kernel<float, false><<<grid, kAppendThreads, 0, s>>>(job);
  }
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
