// fp4_linear.cu -- the product of two matrices in block-scaled 4-bit floating point,
//   out[r][v] = alpha sum_k a[r][k] w[v][k],
// on the fifth-generation tensor cores (tcgen05.mma with block scales): codes and scales go to the
// tensor cores as they are stored, products are exact and summed in fp32, the result is rounded
// once.
//
// The weight's rows are the tile's M (128 per CTA), the activations' rows its N (16 to 192): a head
// has many of the former, a decoding step any number of the latter.  Above 128 activation rows two
// CTAs share a 256-row tile (cta_group::2), each with its half of both operands.  Persistent CTAs,
// K in steps of 256 elements (rows of 128 bytes, four products):
//   warp 0      TMA producer: codes of both operands with the 128-byte swizzle and their scale tiles
//               (512 contiguous bytes each) into a ring of 4 to 10 stages
//   warp 1      copies a stage's scales to tensor memory (tcgen05.cp, ordered before the products that
//               read them) and issues the products into one of two accumulators of 192 columns
//   warps 2-5   epilogue: 32 weight rows a warp, 32 activation rows at a time, transposed in shared memory
//               (stmatrix) and stored in bulk
// Where weight rows are few, clusters share a tile's K instead and join in shared memory (kSplit).
// Every wait on a barrier in shared memory is bounded; a tile whose accumulator does not come is
// written as NaN.
//
// What bounds it (GB300, 128256 x 4096): up to 128 rows the weight's bytes (one row nv, 295 MB: 48
// us, 6.1 TB/s, 90 % of the copy bandwidth; 128 rows mx 50 us), from there the tensor cores: 3840
// rows mx 575 to 600 us, 6.7 to 7.0 PFLOP/s; on 16384 weight rows the tensor pipe is 71 % active in mx
// and 67 % in nv.  With K = 64 to 256 the epilogue does (3840 x 32000: bf16 76 us, f32 93).  What it took: the
// issuing warp whole and its descriptors in uniform registers (issuing a stage took 500 cycles, its
// products take 390), low words of descriptors computed once a stage (nv 99 -> 86 us at 3840 x
// 16384 x 4096), the transposed epilogue (two-byte stores by lane: 1152 us instead of 983 then).
// No gain: scales copied a stage ahead of the products (124 us instead of 99), peeking at the next
// stage's barrier, longer suspensions in waits; in the epilogue the next columns' loads ahead of the
// stores, four staging buffers a warp, rows of 128 bytes by two warps (85.2 us instead of 85.4).
#include <cuda.h>

#include <cuda_bf16.h>

#include "fp4.cuh"
#include "tcgen05.cuh"
#include "tensormap.cuh"

namespace svk {

namespace {

constexpr int kFlM = 128;        // weight rows of a CTA's tile
constexpr int kFlMaxN = 192;     // activation rows of a tile
constexpr int kFlK = 256;        // elements of a stage
constexpr int kFlMaxStages = 10;
constexpr int kFlThreads = 192;
constexpr int kFlMaxSplit = 8;
constexpr int kFlSplitCtas = 128;  // in clusters of eight, as whole clusters fit the chip's GPCs
constexpr uint32_t kFlABytes = kFlM * kFlK / 2;
constexpr uint32_t kFlSfCol = 2 * kFlMaxN;  // first tensor-memory column of the scales
constexpr uint32_t kFlSfBuf = 64;           // columns of one of the two buffers
constexpr uint32_t kFlSfB = 16;             // the activations' scales in a buffer
constexpr size_t kFlSmemMax = 224 * 1024;

template <spec_fp4_format F>
struct Fmt;
template <>
struct Fmt<SPEC_FP4_MX> {
  static constexpr int kGroups = 2;  // scale tiles along a stage
};
template <>
struct Fmt<SPEC_FP4_NV> {
  static constexpr int kGroups = 4;
};

// Instruction descriptor of the block-scaled 4-bit kinds: both operands e2m1 and K-major, scale
// type (ue8m0 or ue4m3), M, N, and which of a tensor-memory word's scales the product starts at.
template <spec_fp4_format F>
__device__ __forceinline__ uint32_t fp4_idesc(int m, int n, int sf) {
  return (1u << 7) | (1u << 10) | ((uint32_t)sf << 4) | ((uint32_t)(n >> 3) << 17) |
         ((F == SPEC_FP4_MX ? 1u : 0u) << 23) | ((uint32_t)(m >> 4) << 24) | ((uint32_t)sf << 29);
}
// Shared-memory descriptors, of which the low word changes from one to the next (by bytes / 16):
// scales, 32 rows of 16 bytes without a swizzle, 8-row groups 128 bytes apart; codes, rows of 128
// bytes with that swizzle (sw128_tile).
constexpr uint32_t kScaleDescHigh = (128u >> 4) | (1u << 14);
constexpr uint32_t kCodeDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kCodeDescLow = (16u >> 4) << 16;

template <int CG, spec_fp4_format F>
__device__ __forceinline__ void fp4_mma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                        uint32_t sfa, uint32_t sfb, bool accumulate) {
#define SVK_FP4_MMA(GROUP, KIND)                                                               \
  asm volatile("{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %6, 0;\n"                \
               " mov.b64 x, {%1, %7};\n mov.b64 y, {%2, %7};\n"                               \
               " tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], x, y, %3, [%4], [%5], p;\n}\n" \
               ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(sfa), "r"(sfb),                       \
               "r"((uint32_t)accumulate), "n"(kCodeDescHigh)                                   \
               : "memory")
  if constexpr (F == SPEC_FP4_MX) {
    if constexpr (CG == 1) SVK_FP4_MMA("1", "mxf4.block_scale.scale_vec::2X");
    else SVK_FP4_MMA("2", "mxf4.block_scale.scale_vec::2X");
  } else {
    if constexpr (CG == 1) SVK_FP4_MMA("1", "mxf4nvf4.block_scale.scale_vec::4X");
    else SVK_FP4_MMA("2", "mxf4nvf4.block_scale.scale_vec::4X");
  }
#undef SVK_FP4_MMA
}
template <int CG>
__device__ __forceinline__ void scales_to_tmem(uint32_t d, uint32_t desc) {
  if constexpr (CG == 1)
    asm volatile("{\n .reg .b64 x;\n mov.b64 x, {%1, %2};\n tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], x;\n}\n" ::"r"(d),
                 "r"(desc), "n"(kScaleDescHigh)
                 : "memory");
  else
    asm volatile("{\n .reg .b64 x;\n mov.b64 x, {%1, %2};\n tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], x;\n}\n" ::"r"(d),
                 "r"(desc), "n"(kScaleDescHigh)
                 : "memory");
}
// Arrives on the barrier (both CTAs' at CG 2) once the products issued so far are done.
template <int CG>
__device__ __forceinline__ void fp4_commit(uint64_t* bar) {
  if constexpr (CG == 1)
    tc05_commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], "
        "%1;\n" ::"r"(smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}
template <int CG>
__device__ __forceinline__ void fp4_alloc(uint32_t* smem_addr) {
  if constexpr (CG == 1) {
    tc05_alloc(smem_addr, 512);
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(
                     smem_u32(smem_addr))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void fp4_dealloc(uint32_t tmem) {
  if constexpr (CG == 1)
    tc05_dealloc(tmem, 512);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;\n" ::"r"(tmem) : "memory");
}
// A box of a tensor map into this CTA's shared memory; its bytes count on `bar`, the address of a
// barrier in this CTA or (CG 2) in the pair's first.
template <int CG>
__device__ __forceinline__ void fp4_load(uint32_t dst, const CUtensorMap* tm, int x, int y, uint32_t bar) {
  if constexpr (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
        "{%2, %3}], [%4];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], "
        "[%1, {%2, %3}], [%4];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ uint32_t first_cta(const void* p) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, 0;\n" : "=r"(a) : "r"(smem_u32(p)));
  return a;
}
template <int CG>
__device__ __forceinline__ void arrive_first(uint64_t* bar) {
  if constexpr (CG == 1)
    mbar_arrive(bar);
  else
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(first_cta(bar))
                 : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

// The epilogue takes 32 columns (activation rows) of its 32 lanes (weight rows) at a time, leaves
// them in shared memory as 32 rows of 32 results side by side, and a bulk store takes them out,
// clipped to the matrix.
template <typename O>
__host__ __device__ constexpr uint32_t out_stage_bytes() {
  return 32 * 32 * sizeof(O);
}
// bf16: pieces of 16 lanes by 8 columns, as the transposing stmatrix wants them (a register pair is
// two columns of one lane); x[0..15] lanes 0..15, x[16..31] lanes 16..31.  fp32: a lane's 32
// columns.
template <typename O>
__device__ __forceinline__ void load_out(uint32_t taddr, uint32_t (&x)[32]) {
  if constexpr (sizeof(O) == 2) {
    tc05_ld_pieces(taddr, x);
    tc05_ld_pieces(taddr + (16u << 16), x + 16);
  } else {
    tc05_ld32(taddr, x);
  }
}
template <typename O>
__device__ __forceinline__ void stage_out(uint32_t buf, int lane, const uint32_t (&x)[32], float alpha,
                                          bool lost) {
  float y[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) y[i] = lost ? CUDART_NAN_F : __uint_as_float(x[i]) * alpha;
  if constexpr (sizeof(O) == 2) {
    // four 8 x 8 pieces a store: lane l gives the place of 8 weight rows (l / 8) in row l % 8; the
    // 16-byte units of the 64-byte rows are swizzled as the bulk store's map says
    const uint32_t at = buf + (uint32_t)(lane & 7) * 64 + (uint32_t)(((lane >> 3) ^ ((lane & 7) >> 1)) << 4);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      uint32_t h[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const __nv_bfloat162 b =
            __floats2bfloat162_rn(y[(q >> 1) * 16 + 4 * g + 2 * (q & 1)], y[(q >> 1) * 16 + 4 * g + 2 * (q & 1) + 1]);
        h[q] = *reinterpret_cast<const uint32_t*>(&b);
      }
      asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};\n" ::"r"(
                       at + (uint32_t)g * 512),
                   "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                   : "memory");
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      asm volatile("st.shared.f32 [%0], %1;\n" ::"r"(buf + (uint32_t)(i * 128 + lane * 4)), "f"(y[i]) : "memory");
  }
}
// Element (column i, weight row j) of a staging buffer.
template <typename O>
__device__ __forceinline__ O staged(uint32_t buf, int i, int j) {
  if constexpr (sizeof(O) == 2) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];\n"
                 : "=h"(v)
                 : "r"(buf + (uint32_t)(i * 64 + (((j >> 3) ^ ((i >> 1) & 3)) << 4) + (j & 7) * 2))
                 : "memory");
    return v;
  } else {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(v) : "r"(buf + (uint32_t)(i * 128 + j * 4)) : "memory");
    return v;
  }
}
__device__ __forceinline__ void bulk_store(const CUtensorMap* tm, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n" ::"l"(
                   reinterpret_cast<uint64_t>(tm)),
               "r"(x), "r"(y), "r"(src)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
}
// A piece that leaves without a bulk store commits an empty group in its place.
__device__ __forceinline__ void bulk_none() {
  asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
}
template <int N>
__device__ __forceinline__ void bulk_store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;\n" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_store_wait() {
  asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
}

// A bounded wait that reads the timer, which takes longer than a stage, only once the barrier has
// been tried often (4096 attempts take 15 ms when nothing comes, and the limit starts after them).
__device__ __forceinline__ bool fp4_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
#pragma unroll 1
  for (int i = 0; i < 4096; ++i)
    if (mbar_try(bar, parity)) return true;
  return mbar_wait(bar, parity, limit_ns);
}

// A place in the ring of stages.
struct Ring {
  int s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++s == stages) {
      s = 0;
      phase ^= 1u;
    }
  }
};

// Four floats at a shared-memory address of CTA `cta` of the cluster, and of this one.
__device__ __forceinline__ void put_four(uint32_t addr, uint32_t cta, const uint32_t* x) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(a) : "r"(addr), "r"(cta));
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(a), "r"(x[0]), "r"(x[1]), "r"(x[2]),
               "r"(x[3])
               : "memory");
}
__device__ __forceinline__ void put_word(const void* p, uint32_t cta, uint32_t x) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(a) : "r"(smem_u32(p)), "r"(cta));
  asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(a), "r"(x) : "memory");
}
__device__ __forceinline__ float4 get_four(uint32_t addr) {
  float4 x;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];\n"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
               : "r"(addr)
               : "memory");
  return x;
}

struct LinearJob {
  int R, V;
  int m_tiles, n_tiles, tile_n;
  int split;              // CTAs of a cluster that share a tile's K (kSplit)
  int k_steps, last_mma;  // stages along K, products of the last one
  int groups;             // scale tiles along K
  int sf_chunks;          // row tiles of the activations' scales that a tile's rows touch
  int stages;
  uint32_t b_bytes;       // of a stage's activations in one CTA
  float alpha;
  void* out;
  int64_t pitch;
  uint64_t wait_limit_ns;
  int stall;              // the tile whose last stage does not come (-1: none; the wait limits' self-test)
};

struct LinearShared {
  uint64_t full[kFlMaxStages], empty[kFlMaxStages], tfull[2], tempty[2];
  uint32_t tmem, lost;  // lost: a part of the tile did not come (kSplit)
};

template <int CG, spec_fp4_format F, typename O, bool kSplit>
__global__ void __launch_bounds__(kFlThreads, 1)
    fp4_linear_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_a,
                      const __grid_constant__ CUtensorMap tm_ws,
                      const __grid_constant__ CUtensorMap tm_as,
                      const __grid_constant__ CUtensorMap tm_out, LinearJob job) {
  constexpr int kGroups = Fmt<F>::kGroups;
  constexpr uint32_t kSfaBytes = kGroups * kScaleTile;
  constexpr uint32_t kStageOut = out_stage_bytes<O>();
  __shared__ LinearShared sh;
  extern __shared__ unsigned char fl_dyn[];
  const uint32_t base = (smem_u32(fl_dyn) + 1023u) & ~1023u;
  const uint32_t stage_bytes =
      kFlABytes + job.b_bytes + kSfaBytes + (uint32_t)job.sf_chunks * kSfaBytes;
  const uint32_t stage_pitch = (stage_bytes + 1023u) & ~1023u;
  // as a uniform value, so that the roles' loops keep descriptors and addresses in uniform
  // registers
  const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int rank = CG == 1 ? 0 : (int)(blockIdx.x & 1u);
  const int share = kSplit ? job.split : CG;  // CTAs of a tile
  const int group = (int)blockIdx.x / share, n_groups = (int)gridDim.x / share;
  // the stages along K that this CTA takes
  const int part = kSplit ? (int)blockIdx.x % job.split : 0;
  const int k0 = kSplit ? job.k_steps * part / job.split : 0;
  const int k1 = kSplit ? job.k_steps * (part + 1) / job.split : job.k_steps;
  const int tiles = job.m_tiles * job.n_tiles;
  const uint64_t limit = job.wait_limit_ns;
  const int stages = job.stages;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&sh.tfull[a], 1);
      mbar_init(&sh.tempty[a], 4 * CG);
    }
    sh.lost = 0u;
    fence_barrier_init();
  }
  if (warp == 1) fp4_alloc<CG>(&sh.tmem);
  tc05_fence_before();
  __syncthreads();
  if (CG > 1) cluster_sync();
  tc05_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)sh.tmem);
  // up to here the launch may overlap the end of the one before it, whose results are read from
  // here on
  asm volatile("griddepcontrol.wait;\n" ::: "memory");

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    Ring ring;
    int filled = 0;
    bool stop = false;
    for (int t = group; t < tiles && !stop; t += n_groups) {
      const int n0 = (t % job.n_tiles) * job.tile_n;
      const int n = min(job.tile_n, (job.R - n0 + 15) & ~15);
      const int row_w = ((t / job.n_tiles) * CG + rank) * kFlM, row_a = n0 + rank * (n / CG);
      const int tile_w = (row_w >> 7) * job.groups, tile_a = (n0 >> 7) * job.groups;
      const bool stall = t == job.stall && (!kSplit || part + 1 == job.split);
      const int k_end = k1 - (stall ? 1 : 0);
      stop = stall;
      for (int kb = k0; kb < k_end; ++kb, ring.next(stages)) {
        if (!__all_sync(kFull, fp4_wait(&sh.empty[ring.s], ring.phase ^ 1u, limit))) {
          stop = true;
          break;
        }
        filled = min(filled + 1, stages);
        const uint32_t a = base + (uint32_t)ring.s * stage_pitch;
        const uint32_t sf = a + kFlABytes + job.b_bytes;
        const uint32_t bar = CG == 1 ? smem_u32(&sh.full[ring.s]) : first_cta(&sh.full[ring.s]);
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&sh.full[ring.s], CG * stage_bytes);
          fp4_load<CG>(a, &tm_w, kb * (kFlK / 2), row_w, bar);
          fp4_load<CG>(a + kFlABytes, &tm_a, kb * (kFlK / 2), row_a, bar);
          fp4_load<CG>(sf, &tm_ws, 0, tile_w + kb * kGroups, bar);
          fp4_load<CG>(sf + kSfaBytes, &tm_as, 0, tile_a + kb * kGroups, bar);
          if (job.sf_chunks > 1)
            fp4_load<CG>(sf + 2 * kSfaBytes, &tm_as, 0, tile_a + job.groups + kb * kGroups, bar);
        }
        __syncwarp();
      }
    }
    // the last stages' products are done, and with them their copies
    if (filled < stages) ring = Ring();
    for (int h = 0; h < filled; ++h, ring.next(stages))
      if (!__all_sync(kFull, fp4_wait(&sh.empty[ring.s], filled < stages ? 0u : ring.phase ^ 1u, limit))) break;
  } else if (warp == 1 && rank == 0) {
    // ---------------- products ----------------
    Ring ring;
    uint32_t lt = 0, it = 0;
    const uint32_t sf_col = tmem + kFlSfCol;  // a multiple of both buffers
    bool stop = false;
    for (int t = group; t < tiles && !stop; t += n_groups, ++lt) {
      const int acc = (int)(lt & 1u);
      if (!__all_sync(kFull, fp4_wait(&sh.tempty[acc], ((lt >> 1) & 1u) ^ 1u, limit))) break;
      tc05_fence_after();
      const int n0 = (t % job.n_tiles) * job.tile_n;
      const int n = min(job.tile_n, (job.R - n0 + 15) & ~15);
      const uint32_t d = tmem + (uint32_t)(acc * kFlMaxN);
      const uint32_t off_b = (uint32_t)(n0 & 127) >> 5;
      const uint32_t idesc0 = fp4_idesc<F>(kFlM * CG, n, 0), idesc2 = fp4_idesc<F>(kFlM * CG, n, 2);
      // the products of a stage; of the last one those that K reaches.  `step`: columns of a
      // group's activation scales.  The next 64 elements are 32 bytes further along the swizzled
      // rows.
      auto issue = [&](uint32_t d, uint32_t a, uint32_t sfa, uint32_t sfb, int step, int kb) {
        const uint32_t b = a + (kFlABytes >> 4);
        const int products = kb + 1 == job.k_steps ? job.last_mma : 4;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j < products) {
            const int g = F == SPEC_FP4_MX ? j >> 1 : j;
            fp4_mma<CG, F>(d, (a + j * 2) | kCodeDescLow, (b + j * 2) | kCodeDescLow,
                           F == SPEC_FP4_MX && (j & 1) ? idesc2 : idesc0, sfa + g * 4, sfb + g * step,
                           kb != k0 || j != 0);
          }
        }
      };
      for (int kb = k0; kb < k1; ++kb, ring.next(stages), ++it) {
        const int s = ring.s;
        if (!__all_sync(kFull, fp4_wait(&sh.full[s], ring.phase, limit))) {
          stop = true;
          break;
        }
        tc05_fence_after();
        const uint32_t a = (base + (uint32_t)s * stage_pitch) >> 4;
        const uint32_t sf = a + ((kFlABytes + job.b_bytes) >> 4);
        const uint32_t sfa = sf_col ^ ((it & 1u) * kFlSfBuf), sfb = sfa + kFlSfB;
        if (elect_one()) {
#pragma unroll
          for (int g = 0; g < kGroups; ++g) scales_to_tmem<CG>(sfa + g * 4, sf + g * (kScaleTile >> 4));
          if (job.sf_chunks == 1) {
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
              scales_to_tmem<CG>(sfb + g * 4, sf + (kGroups + g) * (kScaleTile >> 4));
            issue(d, a, sfa, sfb + off_b, 4, kb);
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int g = 0; g < kGroups; ++g)
                scales_to_tmem<CG>(sfb + (g * 2 + j) * 4, sf + ((1 + j) * kGroups + g) * (kScaleTile >> 4));
            issue(d, a, sfa, sfb + off_b, 8, kb);
          }
          fp4_commit<CG>(&sh.empty[s]);
          if (kb + 1 == k1) fp4_commit<CG>(&sh.tfull[acc]);
        }
        __syncwarp();
      }
    }
  } else if (warp >= 2 && !kSplit) {
    // ---------------- epilogue ----------------
    const int quarter = warp & 3;  // this warp's lanes of tensor memory, 32 of the tile's weight rows
    const uint32_t staging = base + (uint32_t)stages * stage_pitch + (uint32_t)quarter * 2 * kStageOut;
    uint32_t lt = 0, chunk = 0;
    bool lost = false;
    for (int t = group; t < tiles; t += n_groups, ++lt) {
      const int acc = (int)(lt & 1u);
      if (!lost) lost = !__all_sync(kFull, fp4_wait(&sh.tfull[acc], (lt >> 1) & 1u, limit));
      tc05_fence_after();
      const int n0 = (t % job.n_tiles) * job.tile_n, rows = min(job.tile_n, job.R - n0);
      const int v0 = ((t / job.n_tiles) * CG + rank) * kFlM + quarter * 32;
      const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * kFlMaxN);
#pragma unroll 1
      for (int c0 = 0; c0 < rows; c0 += 32, ++chunk) {
        const uint32_t buf = staging + (chunk & 1u) * kStageOut;
        // every piece commits one group: with the newest alone pending, the last store from this
        // buffer has read it
        if (lane == 0) bulk_store_wait_read<1>();
        __syncwarp();
        uint32_t x[32];
        load_out<O>(taddr + (uint32_t)c0, x);
        tc05_wait_ld();
        tc05_landed(x);
        if (c0 + 32 >= rows) {  // the accumulator may be written again
          tc05_fence_before();
          __syncwarp();
          if (lane == 0) arrive_first<CG>(&sh.tempty[acc]);
        }
        stage_out<O>(buf, lane, x, job.alpha, lost);
        if (v0 + 32 <= job.V) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) bulk_store(&tm_out, buf, v0, n0 + c0);
        } else {  // a bulk store clips to 16 bytes, the matrix may end within them
          if (lane == 0) bulk_none();
          __syncwarp();
          if (v0 + lane < job.V)
            for (int i = 0; i < min(32, rows - c0); ++i)
              static_cast<O*>(job.out)[(int64_t)(n0 + c0 + i) * job.pitch + v0 + lane] = staged<O>(buf, i, lane);
          __syncwarp();
        }
      }
    }
    if (lane == 0) bulk_store_wait();
  }
  if constexpr (kSplit) {
    // The parts of a tile along K are joined in shared memory, which the stages no longer need:
    // every CTA of the cluster owns an equal run of the activations' rows, in fours, and gets the
    // others' parts of them. One tile per cluster.  A CTA whose products did not come tells all: its
    // copies may still be on their way to the memory where the parts are joined.
    const int quarter = warp & 3, n = job.R, own = (n + 4 * job.split - 1) / (4 * job.split);  // fours
    const int lane_v = quarter * 32 + lane, v = group * kFlM + lane_v;
    bool lost = false;
    __syncwarp();
    if (warp >= 2) lost = !__all_sync(kFull, fp4_wait(&sh.tfull[0], 0u, limit));
    cluster_sync();  // all products of the tile are done
    if (lost && lane == 0)
      for (int q = 0; q < job.split; ++q) put_word(&sh.lost, (uint32_t)q, 1u);
    if (warp >= 2) {
      tc05_fence_after();
#pragma unroll 1
      for (int c0 = 0; c0 < n; c0 += 32) {
        uint32_t x[32];
        tc05_ld32(tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)c0, x);
        tc05_wait_ld();
        tc05_landed(x);
        int owner = c0 / 4 / own, four = c0 / 4 % own;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (c0 + 4 * i < n) {
            put_four(base + (uint32_t)((part * own + four) * kFlM + lane_v) * 16, (uint32_t)owner, x + 4 * i);
            if (++four == own) {
              four = 0;
              ++owner;
            }
          }
        }
      }
      tc05_fence_before();
    }
    __syncwarp();
    cluster_sync();  // the parts are there
    if (warp >= 2 && v < job.V) {
      const int row0 = part * own * 4;
      const float alpha = *reinterpret_cast<volatile uint32_t*>(&sh.lost) ? CUDART_NAN_F : job.alpha;
      for (int four = 0; four < own && row0 + four * 4 < n; ++four) {
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int q = 0; q < job.split; ++q) {
          const float4 x = get_four(base + (uint32_t)((q * own + four) * kFlM + lane_v) * 16);
          y.x += x.x;
          y.y += x.y;
          y.z += x.z;
          y.w += x.w;
        }
        const float z[4] = {y.x, y.y, y.z, y.w};
        O* out = static_cast<O*>(job.out) + (int64_t)(row0 + four * 4) * job.pitch + v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (row0 + four * 4 + i < n) {
            if constexpr (sizeof(O) == 2)
              reinterpret_cast<__nv_bfloat16*>(out)[i * job.pitch] = __float2bfloat16_rn(z[i] * alpha);
            else
              out[i * job.pitch] = z[i] * alpha;
          }
        }
      }
    }
  }
  __syncwarp();
  tc05_fence_before();
  __syncthreads();
  if (CG > 1) cluster_sync();
  tc05_fence_after();
  if (warp == 1) fp4_dealloc<CG>(tmem);
}

// Rows of codes, boxes of 128 bytes by box_rows.
bool code_map(CUtensorMap* map, const void* p, int rows, int64_t row_bytes, int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)row_bytes, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
  const cuuint32_t box[2] = {kFlK / 2, (cuuint32_t)box_rows};
  const cuuint32_t one[2] = {1, 1};
  return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(p), dims, strides, box, one,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Scale tiles one after another, boxes of `n` of them.
bool scale_map(CUtensorMap* map, const void* p, int64_t tiles, int n) {
  const cuuint64_t dims[2] = {kScaleTile / 4, (cuuint64_t)tiles};
  const cuuint64_t strides[1] = {kScaleTile};
  const cuuint32_t box[2] = {kScaleTile / 4, (cuuint32_t)n};
  const cuuint32_t one[2] = {1, 1};
  return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(p), dims, strides, box, one,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The result, boxes of 32 x 32, rows of 64 bytes with that swizzle or of 128 bytes without one.
template <typename O>
bool out_map(CUtensorMap* map, void* p, int R, int V, int64_t pitch) {
  constexpr bool kHalf = sizeof(O) == 2;
  const cuuint64_t dims[2] = {(cuuint64_t)V, (cuuint64_t)R};
  const cuuint64_t strides[1] = {(cuuint64_t)pitch * sizeof(O)};
  const cuuint32_t box[2] = {32, 32};
  const cuuint32_t one[2] = {1, 1};
  return encode_fn()(map, kHalf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, p,
                     dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     kHalf ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE,
                     CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int CG, spec_fp4_format F, typename O, bool kSplit = false>
cudaError_t launch_linear(const void* a, const void* a_scales, const void* w, const void* w_scales,
                          int K, LinearJob job, cudaStream_t s) {
  if (!encode_fn()) return cudaErrorNotSupported;
  constexpr int kGroups = Fmt<F>::kGroups;
  const int64_t row_bytes = fp4_row_bytes(K);
  job.groups = fp4_groups(K, F);
  job.k_steps = (int)((row_bytes * 2 + kFlK - 1) / kFlK);
  job.last_mma = (int)((row_bytes * 2 - (int64_t)(job.k_steps - 1) * kFlK + 63) / 64);
  job.m_tiles = (job.V + CG * kFlM - 1) / (CG * kFlM);
  const int box_n = (job.tile_n / CG + 7) & ~7;
  job.b_bytes = (uint32_t)box_n * (kFlK / 2);
  const uint32_t stage = (kFlABytes + job.b_bytes + (uint32_t)((1 + job.sf_chunks) * kGroups * kScaleTile) +
                          1023u) & ~1023u;
  constexpr uint32_t kStaging = 4 * 2 * out_stage_bytes<O>();  // two buffers per epilogue warp
  job.stages = (int)((kFlSmemMax - 1024 - kStaging) / stage);
  if (job.stages > kFlMaxStages) job.stages = kFlMaxStages;
  const size_t smem = 1024 + (size_t)job.stages * stage + kStaging;
  CUtensorMap tm_w, tm_a, tm_ws, tm_as, tm_out;
  if (!code_map(&tm_w, w, job.V, row_bytes, kFlM) || !code_map(&tm_a, a, job.R, row_bytes, box_n) ||
      !scale_map(&tm_ws, w_scales, (int64_t)fp4_row_tiles(job.V) * job.groups, kGroups) ||
      !scale_map(&tm_as, a_scales, (int64_t)fp4_row_tiles(job.R) * job.groups, kGroups) ||
      !out_map<O>(&tm_out, job.out, job.R, job.V, job.pitch))
    return cudaErrorInvalidValue;
  auto kernel = fp4_linear_kernel<CG, F, O, kSplit>;
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kFlSmemMax);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev] = true;
  }
  int64_t groups = device_sm_count() / CG;
  if (groups > (int64_t)job.m_tiles * job.n_tiles) groups = (int64_t)job.m_tiles * job.n_tiles;
  const int cluster = kSplit ? job.split : CG;
  if (kSplit) groups = job.m_tiles;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(groups * cluster));
  cfg.blockDim = dim3(kFlThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, tm_w, tm_a, tm_ws, tm_as, tm_out, job);
}

template <spec_fp4_format F, typename O>
cudaError_t launch_linear_group(const void* a, const void* a_scales, const void* w, const void* w_scales,
                                int K, LinearJob job, cudaStream_t s) {
  // Few weight rows: clusters of up to eight CTAs share a tile's K, two stages each at least, where
  // that many are resident at once and what it saves, a quarter of a microsecond a stage, is more
  // than the join costs, one and a thirtieth per activation row.  Measured (us, mx, shared and
  // not): 1 x 4096 x 4096 5.1 and 6.6, 60 x 4096 x 8192 7.9 and 10.7, 1 x 4096 x 14336 7.5 and
  // 15.4, 192 x 4096 x 14336 14.6 and 18.3; but 128 x 4096 x 4096 9.2 and 8.6, 64 x 8192 x 4096 8.2
  // and 7.2.
  const int tiles = (job.V + kFlM - 1) / kFlM, steps = (int)((fp4_row_bytes(K) * 2 + kFlK - 1) / kFlK);
  job.split = 1;
  while (job.split < kFlMaxSplit && tiles * job.split * 2 <= kFlSplitCtas && steps >= job.split * 4)
    job.split *= 2;
  if (job.n_tiles == 1 && 7 * (int64_t)steps * (job.split - 1) >= (int64_t)job.split * (30 + job.R))
    return launch_linear<1, F, O, true>(a, a_scales, w, w_scales, K, job, s);
  // Pairs of CTAs halve the reads of the activations; below, the weight's bytes bound both and
  // single CTAs start sooner.  Measured on 128256 x 4096 (us, mx, pairs and not): 60 rows 51.3 and
  // 48.0, 128 rows 52.1 and 51.4, 192 rows 54.8 and 57.9, 3840 rows 576 and 710.
  if (job.R > 128) return launch_linear<2, F, O>(a, a_scales, w, w_scales, K, job, s);
  return launch_linear<1, F, O>(a, a_scales, w, w_scales, K, job, s);
}

}  // namespace

cudaError_t launch_fp4_linear(const void* a_codes, const void* a_scales, const void* w_codes,
                              const void* w_scales, spec_fp4_format format, int R, int V, int K,
                              float alpha, void* out, spec_dtype dtype, int64_t pitch, int stall,
                              cudaStream_t s) {
  LinearJob job{};
  job.R = R;
  job.V = V;
  job.alpha = alpha;
  job.out = out;
  job.pitch = pitch;
  job.wait_limit_ns = stall >= 0 ? 20000000ull : 2000000000ull;
  job.stall = stall;
  // tiles of equal numbers of rows; more than one start at multiples of 64 rows, where the scales'
  // columns in tensor memory are aligned
  job.n_tiles = (R + kFlMaxN - 1) / kFlMaxN;
  const int per = (R + job.n_tiles - 1) / job.n_tiles;
  job.tile_n = job.n_tiles == 1 ? (per + 15) & ~15 : (per + 63) & ~63;
  job.n_tiles = (R + job.tile_n - 1) / job.tile_n;
  job.sf_chunks = job.tile_n <= 128 && (job.n_tiles == 1 || 128 % job.tile_n == 0) ? 1 : 2;
  if (format == SPEC_FP4_MX)
    return dtype == SPEC_BF16
               ? launch_linear_group<SPEC_FP4_MX, uint16_t>(a_codes, a_scales, w_codes, w_scales, K, job, s)
               : launch_linear_group<SPEC_FP4_MX, float>(a_codes, a_scales, w_codes, w_scales, K, job, s);
  return dtype == SPEC_BF16
             ? launch_linear_group<SPEC_FP4_NV, uint16_t>(a_codes, a_scales, w_codes, w_scales, K, job, s)
             : launch_linear_group<SPEC_FP4_NV, float>(a_codes, a_scales, w_codes, w_scales, K, job, s);
}

}  // namespace svk

using namespace svk;

namespace {

int linear_call(const void* a_codes, const void* a_scales, const void* w_codes, const void* w_scales,
                spec_fp4_format format, int32_t R, int32_t V, int32_t K, float alpha, void* out,
                spec_dtype dtype, int64_t row_pitch, int32_t stall, spec_stream_t stream) {
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_UNSUPPORTED_DTYPE;
  if (format != SPEC_FP4_MX && format != SPEC_FP4_NV) return SPEC_ERR_UNSUPPORTED_DTYPE;
  if (R < 0 || V < 1 || K < 1 || row_pitch < V) return SPEC_ERR_INVALID_ARG;
  if (!(alpha >= -3.402823466e38f && alpha <= 3.402823466e38f)) return SPEC_ERR_INVALID_ARG;
  if (R > SPEC_FP4_MAX_DIM || V > SPEC_FP4_MAX_DIM || K > SPEC_FP4_MAX_DIM || row_pitch >= (int64_t)1 << 37 ||
      (int64_t)fp4_row_tiles(R > V ? R : V) * fp4_groups(K, format) > INT32_MAX - 8 ||
      ((int64_t)R + 63) / 64 * (((int64_t)V + 127) / 128) > INT32_MAX)
    return SPEC_ERR_TOO_LARGE;
  if (R == 0) return SPEC_OK;
  if (!a_codes || !a_scales || !w_codes || !w_scales || !out) return SPEC_ERR_INVALID_ARG;
  const uintptr_t all = reinterpret_cast<uintptr_t>(a_codes) | reinterpret_cast<uintptr_t>(a_scales) |
                        reinterpret_cast<uintptr_t>(w_codes) | reinterpret_cast<uintptr_t>(w_scales) |
                        reinterpret_cast<uintptr_t>(out);
  if ((all & 15u) || row_pitch * (dtype == SPEC_BF16 ? 2 : 4) % 16 != 0) return SPEC_ERR_MISALIGNED;
  return launch_fp4_linear(a_codes, a_scales, w_codes, w_scales, format, R, V, K, alpha, out, dtype,
                           row_pitch, stall, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SPEC_OK
             : SPEC_ERR_CUDA;
}

}  // namespace

extern "C" int spec_fp4_linear(const void* a_codes, const void* a_scales, const void* w_codes,
                               const void* w_scales, spec_fp4_format format, int32_t R, int32_t V,
                               int32_t K, float alpha, void* out, spec_dtype dtype, int64_t row_pitch,
                               spec_stream_t stream) {
  return linear_call(a_codes, a_scales, w_codes, w_scales, format, R, V, K, alpha, out, dtype, row_pitch,
                     -1, stream);
}

extern "C" int spec_fp4_linear_test_stall(const void* a_codes, const void* a_scales, const void* w_codes,
                                          const void* w_scales, spec_fp4_format format, int32_t R,
                                          int32_t V, int32_t K, float alpha, void* out, spec_dtype dtype,
                                          int64_t row_pitch, int32_t tile, spec_stream_t stream) {
  if (tile < 0) return SPEC_ERR_INVALID_ARG;
  return linear_call(a_codes, a_scales, w_codes, w_scales, format, R, V, K, alpha, out, dtype, row_pitch,
                     tile, stream);
}
