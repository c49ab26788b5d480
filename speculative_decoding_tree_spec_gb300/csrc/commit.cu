// commit.cu -- accepted-path commit: after a verify step, move the cache entries of
// each tree's accepted path to consecutive positions after its prefix, in every
// plane of a strided cache (target or draft KV cache, or the features), so the
// caches continue the accepted sequence ("EAGLE close reading", edgeai1.github.io,
// section 5: both caches are trimmed to what was accepted).
//
// Node n of tree b sits at position prefix_len[b] + n; position prefix_len[b] + k
// receives node path[b][k] for k = 1 .. accept_len[b] (k = 0 is the root, already in
// place).  A path increases strictly (parents precede children), so path[b][k] >= k;
// one thread owns each 16-byte column of a (plane, tree) and no other thread touches
// its bytes.
#include "paged.cuh"

namespace svk {

namespace {

constexpr int kCommitThreads = 256;

struct CommitJob {
  unsigned char* cache;
  int B, n_planes, n_pos, W;
  int64_t plane_stride, batch_stride, pos_stride;  // bytes
  int64_t row_bytes;                               // multiple of 16
  const int32_t* prefix_len;
  const int32_t* path;
  const int32_t* accept_len;
};

constexpr int kBatchMoves = 8;  // moves whose sources one thread loads before storing

// One thread per (plane, tree, 16-byte column) item, grid-stride.  The moves of a tree
// are taken in batches of kBatchMoves in increasing k: a batch loads all its sources,
// then stores all its destinations.  Sources of later batches lie above every
// destination of earlier ones (path[k] >= k), so nothing is read after it is
// overwritten.
__global__ void __launch_bounds__(kCommitThreads) commit_kernel(CommitJob job) {
  const int64_t nvec = job.row_bytes / 16;
  const int64_t total = (int64_t)job.B * job.n_planes * nvec;
  for (int64_t item = (int64_t)blockIdx.x * kCommitThreads + threadIdx.x; item < total;
       item += (int64_t)gridDim.x * kCommitThreads) {
    const int64_t pair = item / nvec, v = item - pair * nvec;
    const int b = (int)(pair % job.B);
    const int plane = (int)(pair / job.B);
    const int a = min(job.accept_len[b], job.W - 1);
    if (a <= 0) continue;
    const int base = job.prefix_len[b];
    const int32_t* path = job.path + (int64_t)b * job.W;
    unsigned char* col = job.cache + plane * job.plane_stride + (int64_t)b * job.batch_stride + v * 16;
    for (int k0 = 1; k0 <= a; k0 += kBatchMoves) {
      uint4 x[kBatchMoves];
      int dst[kBatchMoves];
#pragma unroll
      for (int i = 0; i < kBatchMoves; ++i) {
        const int k = k0 + i;
        dst[i] = -1;
        if (k <= a) {
          const int src = base + path[k], d = base + k;
          if (src != d && src >= 0 && src < job.n_pos && d < job.n_pos) {
            x[i] = *reinterpret_cast<const uint4*>(col + src * job.pos_stride);
            dst[i] = d;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kBatchMoves; ++i)
        if (dst[i] >= 0) *reinterpret_cast<uint4*>(col + dst[i] * job.pos_stride) = x[i];
    }
  }
}

// The same in a paged cache: a position's row is found through the sequence's page table,
// and a row may be split over heads that lie apart.
struct PagedCommitJob {
  unsigned char* cache;
  int n_pages, max_pages, W;
  int items;              // 16-byte columns of a tree: planes * heads * columns of a row
  int blocks_per_tree;
  FastDiv by_vec, by_head;
  int64_t plane_stride, page_stride, pos_stride, head_stride;  // bytes
  PageDiv pd;
  const int32_t* table;
  const int32_t* prefix_len;
  const int32_t* path;
  const int32_t* accept_len;
};

constexpr int kPagedMoves = 4;    // moves of a batch
constexpr int kPagedColumns = 2;  // columns a thread moves at once

// A block takes one tree and some of its columns (every blocks_per_tree-th run).  Its first
// threads find the rows of up to kPagedMoves moves through the page table, once for all
// columns; each thread then loads two columns of every one of them before it stores any.  What
// bounds it is latency, the chain path -> page table -> row -> store: so all blocks are
// resident at once, and a thread has eight loads in flight.  64 planes x 64 trees of 2 KB rows:
// 23.3 us where every thread looked its rows up (a quarter of the threads resident), 16.3 us with
// one column at a time and 3.4 waves of blocks.
__global__ void __launch_bounds__(kCommitThreads, 4) paged_commit_kernel(PagedCommitJob job) {
  __shared__ int64_t src[kPagedMoves], dst[kPagedMoves];
  const int b = blockIdx.x / job.blocks_per_tree, part = blockIdx.x % job.blocks_per_tree;
  const int a = min(job.accept_len[b], job.W - 1);
  const int64_t base = max(job.prefix_len[b], 0);  // as the append that stored the nodes
  const int32_t* path = job.path + (int64_t)b * job.W;
  for (int k0 = 1; k0 <= a; k0 += kPagedMoves) {
    if (threadIdx.x < 2 * kPagedMoves) {
      const int i = threadIdx.x % kPagedMoves, k = k0 + i;
      const int node = k < job.W ? path[k] : 0;  // (read beside accept_len, not after it)
      const bool to = threadIdx.x >= kPagedMoves;
      const int64_t t = base + (to ? k : node);
      int64_t at = -1;
      if (k <= a && node != k && t >= 0 && t <= SPEC_MAX_POSITIONS)
        at = paged_offset(job.table + (int64_t)b * job.max_pages, job.max_pages, job.n_pages,
                          job.pd, job.page_stride, job.pos_stride, (int)t);
      (to ? dst : src)[i] = at;
    }
    __syncthreads();
    constexpr int kRun = kPagedColumns * kCommitThreads;
    for (int run = part * kRun; run < job.items; run += job.blocks_per_tree * kRun) {
      unsigned char* col[kPagedColumns];
      uint4 x[kPagedColumns][kPagedMoves];
#pragma unroll
      for (int c = 0; c < kPagedColumns; ++c) {
        const int item = run + c * kCommitThreads + threadIdx.x;
        const int row = job.by_vec.div(item), plane = job.by_head.div(row);
        col[c] = item < job.items ? job.cache + plane * job.plane_stride +
                                        (row - plane * job.by_head.d) * job.head_stride +
                                        (int64_t)(item - row * job.by_vec.d) * 16
                                  : nullptr;
#pragma unroll
        for (int i = 0; i < kPagedMoves; ++i)
          if (col[c] && src[i] >= 0 && dst[i] >= 0)
            x[c][i] = *reinterpret_cast<const uint4*>(col[c] + src[i]);
      }
#pragma unroll
      for (int c = 0; c < kPagedColumns; ++c)
#pragma unroll
        for (int i = 0; i < kPagedMoves; ++i)
          if (col[c] && src[i] >= 0 && dst[i] >= 0)
            *reinterpret_cast<uint4*>(col[c] + dst[i]) = x[c][i];
    }
    __syncthreads();
  }
}

}  // namespace

}  // namespace svk

using namespace svk;

extern "C" int spec_commit_accepted_path_paged(
    void* cache, int32_t B, int32_t n_planes, int32_t n_heads, int32_t n_pages,
    int32_t page_size, int64_t plane_stride, int64_t page_stride, int64_t pos_stride,
    int64_t head_stride, int64_t row_bytes, const int32_t* page_table, int32_t max_pages,
    const int32_t* prefix_len, const int32_t* accepted_path, const int32_t* accept_len, int32_t W,
    spec_stream_t stream) {
  if (B < 0 || n_planes < 0 || n_heads < 0 || row_bytes < 0 || W < 1 || plane_stride < 0)
    return SPEC_ERR_INVALID_ARG;
  const spec_paged_layout l{n_pages, page_size, 1, 1, page_stride, pos_stride, head_stride};
  const int rc = check_paged_layout(l, max_pages);
  if (rc != SPEC_OK) return rc;
  if (B == 0 || n_planes == 0 || n_heads == 0 || row_bytes == 0) return SPEC_OK;
  if (!cache || !page_table || !prefix_len || !accepted_path || !accept_len)
    return SPEC_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(cache) & 15u) ||
      ((plane_stride | page_stride | pos_stride | head_stride | row_bytes) & 15))
    return SPEC_ERR_MISALIGNED;
  if (row_bytes > pos_stride && page_size > 1) return SPEC_ERR_INVALID_ARG;  // rows may not overlap
  const int64_t nvec = row_bytes / 16;
  if ((int64_t)n_planes * n_heads > 0x3fffffff || nvec > 0x3fffffff ||
      (int64_t)n_planes * n_heads * nvec > 0x3fffffff)
    return SPEC_ERR_TOO_LARGE;
  PagedCommitJob job{};
  job.cache = static_cast<unsigned char*>(cache);
  job.n_pages = n_pages;
  job.max_pages = max_pages;
  job.W = W;
  job.items = (int)(n_planes * n_heads * nvec);
  job.by_vec = FastDiv::make((int)nvec);
  job.by_head = FastDiv::make(n_heads);
  job.plane_stride = plane_stride;
  job.page_stride = page_stride;
  job.pos_stride = pos_stride;
  job.head_stride = head_stride;
  job.pd = PageDiv::make(page_size);
  job.table = page_table;
  job.prefix_len = prefix_len;
  job.path = accepted_path;
  job.accept_len = accept_len;
  // no more blocks than are resident at once, and than there are columns
  const int run = kPagedColumns * kCommitThreads;
  const int runs = (job.items + run - 1) / run;
  const int share = device_sm_count() * 4 / B;
  job.blocks_per_tree = share < 1 ? 1 : share < runs ? share : runs;
  const int64_t blocks = (int64_t)B * job.blocks_per_tree;
  if (blocks > 0x7fffffff) return SPEC_ERR_TOO_LARGE;
  paged_commit_kernel<<<(unsigned)blocks, kCommitThreads, 0,
                        reinterpret_cast<cudaStream_t>(stream)>>>(job);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

extern "C" int spec_commit_accepted_path(void* cache, int32_t B, int32_t n_planes, int32_t n_pos,
                                         int64_t plane_stride, int64_t batch_stride,
                                         int64_t pos_stride, int64_t row_bytes,
                                         const int32_t* prefix_len,
                                         const int32_t* accepted_path,
                                         const int32_t* accept_len, int32_t W,
                                         spec_stream_t stream) {
  if (B < 0 || n_planes < 0 || n_pos < 0 || W < 1 || row_bytes < 0) return SPEC_ERR_INVALID_ARG;
  if (B == 0 || n_planes == 0 || row_bytes == 0) return SPEC_OK;
  if (!cache || !prefix_len || !accepted_path || !accept_len) return SPEC_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(cache) & 15u) || (plane_stride & 15) || (batch_stride & 15) ||
      (pos_stride & 15) || (row_bytes & 15))
    return SPEC_ERR_MISALIGNED;
  if (row_bytes > pos_stride && n_pos > 1) return SPEC_ERR_INVALID_ARG;  // rows may not overlap
  const int64_t pairs = (int64_t)B * n_planes;
  if (pairs > 0x7fffffff) return SPEC_ERR_TOO_LARGE;
  CommitJob job{};
  job.cache = static_cast<unsigned char*>(cache);
  job.B = B;
  job.n_planes = n_planes;
  job.n_pos = n_pos;
  job.W = W;
  job.plane_stride = plane_stride;
  job.batch_stride = batch_stride;
  job.pos_stride = pos_stride;
  job.row_bytes = row_bytes;
  job.prefix_len = prefix_len;
  job.path = accepted_path;
  job.accept_len = accept_len;
  const int64_t items = pairs * (row_bytes / 16);
  int64_t blocks = (items + kCommitThreads - 1) / kCommitThreads;
  const int64_t cap = (int64_t)device_sm_count() * 16;  // grid-stride beyond this
  if (blocks > cap) blocks = cap;
  commit_kernel<<<(unsigned)blocks, kCommitThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(job);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
