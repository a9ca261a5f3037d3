// gemm_block.cu -- matrix products of E4M3 codes with a scale for each block of 128 along K:
//   C[m, n] = sum over 128-wide slices j of K of  (A_j B_j^T)[m, n] / (s_a[j, m] s_b(j, n))  + bias[n]
// A [M, K] and B [N, K] hold codes (rows of lda, ldb bytes), s_a [ceil(K/128), M]; B's scale is one per
// 128 x 128 tile (a weight) or one per row and slice, [ceil(K/128), N] (the second operand of a weight
// gradient).  Each slice's product is a sum of at most 128 products of E4M3 codes in the tensor core's
// float32 accumulator; it is taken out of tensor memory, scaled and added in float32 registers in slice
// order, so the result is the same from call to call.
//
// block_pair_kernel (many rows): 256 x 256 output tiles on CTA pairs (tcgen05 cta_group::2), as in
// gemm_pair.cuh: each CTA stages its 128 rows of A and 128 rows of B, 32 KB per slice.  A slice's product
// is 256 columns of TMEM, so two fit, and a buffer comes back to the MMA only after eight warps have read
// it.  What bounds the kernel is that round trip (MMA, commit, TMEM loads, arrival at the leader: about
// 2000 cycles for two slices of 512 each), so it is cut into halves of 128 columns with an MMA issuer, a
// warpgroup and barriers of their own; the arrivals carry no release at cluster scope, the waits read no
// timer, a warp's scales come through a ring of asynchronous copies, and the issuers run on whole warps.
// Each promotion thread holds a row's 128 float32 sums in registers (setmaxnreg moves them over from the
// other warpgroup); the scales' ring runs on from tile to tile, and the outputs leave through shared memory by
// TMA.  From captured graphs 8192^3 takes 468 us, 2.35 PFLOP/s (480 to 489 back to back), and 4608 x 12288 x 4096 with
// bias 210 us, 2.21 PFLOP/s (launched one by one 219).  When they took 464 and 208, a ring that started anew with each
// tile took 492 and 227 us, with it but each thread storing its own row 472 and 218; at that first step the loop without
// the multiply-adds took 420 and 196 us, without reading TMEM either 332 and 156, with one N = 256 MMA and barrier per
// slice 558 and 256, with barriers for quarters of 64 columns 668 and 299.  The sums and loads fill the 232 registers:
// 12 to 24 bytes of each form are spilled.
//
// block_stream_kernel (tens of rows, or too few tiles for the pairs): B's bytes are the cost, so the roles are
// turned: 128 rows of B are the MMA's M side and 32 or 64 rows of A its N side, four slices' products in TMEM,
// and the CTAs of a cluster split K, so that every SM streams its share of B through a ring of TMA stages.  The
// partial sums meet in shared memory of the cluster (each CTA adds up its own columns, in rank order): no
// workspace, no atomics, the same bits every time.  48 x 4096 x 14336: 18.0 us, 3.3 TB/s (through the ring, behind a
// cluster barrier of its own: 20.2); about 10 us of it are HBM time, the rest launch, first bytes and the join.
//
// block_few_kernel (up to 16 rows): B streams through rings of asynchronous copies that every warp keeps for
// itself, straight into the register layout of mma.sync.  At these sizes the tensor cores' rate does not count
// and the latency does: no TMEM to allocate, no barrier and no cluster between the first copy and the sums.
// 1 x 12288 x 4096: 11.4 us, 4.4 TB/s, of which 2 are the launch; 1 x 1024 x 1024: 2.2 us.
//
// Every wait is bounded (common.cuh); after one gives up the remaining barriers are still met, so no
// thread is left behind.
#include <atomic>

#include "gemm_kernel.cuh"

namespace mmdit {
namespace {

constexpr int kSlice = 128;  // K of a scale block: 128 codes = one 128-byte swizzled row
constexpr int kPairStages = 4;  // what the output boxes leave room for; more only spread the pairs apart in L2
                                // (8192^3 before the boxes: 493 us with 4, 507 with 5, 514 with 6, 522 with 3)
constexpr int kPairStageBytes = 2 * kSlice * kSlice;  // this CTA's 128 rows of A and of B
constexpr int kPairThreads = 128 + 256;               // producer, two MMA issuers, an idle warp; 8 promotion warps
constexpr int kRing = 4, kRingFloats = 32 + 128;      // per promotion warp: slices whose scales are held, floats of one
constexpr int kBox = 32 * 128;                        // an output box: 32 rows of 128 bytes; two per promotion warp
constexpr int kPairSmem = kPairStages * kPairStageBytes + 8 * 2 * kBox + 8 * kRing * kRingFloats * 4 + 256 + 1024;
// 384 threads start with 168 registers (64512); the promotion warpgroups take 232, the other one keeps 40
constexpr int kPairFewRegs = 40, kPairManyRegs = 232;
static_assert(128 * kPairFewRegs + 256 * kPairManyRegs <= kPairThreads * 168, "register shares");
constexpr int kPairN = 256;

// mbar_wait that tries the barrier a few hundred times before it first reads the timer: the waits here
// recur every slice, and a timer read costs more than the slice's hand-over.
__device__ __forceinline__ bool slice_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* status) {
#pragma unroll 1
  for (int i = 0; i < 256; ++i)
    if (mbar_test(bar, parity)) return true;
  return mbar_wait(bar, parity, abort, status, kErrGemmWait);
}

// slice_wait by a whole warp, with one answer for all lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* status) {
  return __all_sync(0xffffffffu, slice_wait(bar, parity, abort, status)) != 0;
}

// One lane of a converged warp.  The MMA and TMA loops below run on whole warps and let one lane issue:
// descriptors and counters then stay in uniform registers, which a loop that only one lane walks cannot
// use (each MMA would first move its operands there: 450 instead of 100 cycles for a slice's four).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Four bytes copied to shared memory while the thread goes on; groups of them are awaited in order.
__device__ __forceinline__ void copy_async4(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes, or zeros where `ok` is false (the source is then not read).
__device__ __forceinline__ void copy_async16(uint32_t dst, const uint8_t* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Moves registers between the warpgroups of a CTA: the sum of the shares is what the launch gave.
template <int R>
__device__ __forceinline__ void regs_more() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void regs_fewer() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// A box of shared memory stored to the tensor at column x, row y while the thread goes on; groups of stores are
// awaited in order: until their shared memory is read, or until they are done.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* tm, const void* box, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(tm), "r"(smem_addr(box)),
               "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void store_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }
template <int N>
__device__ __forceinline__ void store_wait() { asm volatile("cp.async.bulk.wait_group %0;" ::"n"(N) : "memory"); }

// 64 columns of 16 lanes of this warp's quarter: lane 4 g + q receives columns 8 i + 2 q, 8 i + 2 q + 1 of row g in
// r[4 i], r[4 i + 1] and of row g + 8 in r[4 i + 2], r[4 i + 3].
__device__ __forceinline__ void tmem_ld16x64(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

struct BlockArgs {
  const float* sa;   // [num_kb, M]
  const float* sb;   // tile scales: (n / 128) * sb_n + kb * sb_k; row scales: kb * N + n
  int64_t sb_n, sb_k;
  const __nv_bfloat16* bias;
  void* out;         // [M, N]
  int M, N, num_kb;
  uint32_t* status;
  int clear;         // 1: this kernel is the call's first and clears the status word
};

template <typename TO>
__device__ __forceinline__ void store_row(TO* dst, const __nv_bfloat16* bias, int n, int N, float (&v)[32]) {
  if (n + 32 <= N) {
    if (bias) {
      float b[32];
      load32(bias + n, b);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] += b[i];
    }
    store32(dst + n, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    if (n + i < N) {
      const float r = v[i] + (bias ? __bfloat162float(bias[n + i]) : 0.f);
      if constexpr (sizeof(TO) == 2)
        dst[n + i] = __float2bfloat16(r);
      else
        dst[n + i] = r;
    }
  }
}

// ----------------------------------------------------------------------------- many rows
template <bool ROW_B, typename TO, int SPLITS>
__global__ void __cluster_dims__(2 * SPLITS, 1, 1) __launch_bounds__(kPairThreads, 1)
    block_pair_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                      const __grid_constant__ CUtensorMap tm_out, const __grid_constant__ BlockArgs a) {
  constexpr uint32_t kIdesc = make_idesc<kKindF8>(256, 128);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* boxes = smem + kPairStages * kPairStageBytes;                     // [8 warps][2][kBox]
  float* rings = reinterpret_cast<float*>(boxes + 8 * 2 * kBox);             // [8 warps][kRing][kRingFloats]
  uint64_t* full = reinterpret_cast<uint64_t*>(rings + 8 * kRing * kRingFloats);
  uint64_t* empty = full + kPairStages;
  uint64_t* pfull = empty + kPairStages;  // [buffer][half]
  uint64_t* pempty = pfull + 4;
  uint64_t* drain = pempty + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  // a cluster is SPLITS (1 or 2) pairs, which share a tile's K: CTA `rank` of pair `part`
  const uint32_t cta = cluster_ctarank(), rank = cta & 1, lead = SPLITS > 1 ? cta & ~1u : 0;
  const uint16_t both = static_cast<uint16_t>(3u << lead);
  const int part = SPLITS > 1 ? static_cast<int>(cta >> 1) : 0;
  const bool leader = rank == 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int first = (a.num_kb + SPLITS - 1) / SPLITS;  // slices of pair 0
  const int kb0 = part * first, num_kb = part ? a.num_kb - first : first;
  const int tiles_m = (a.M + 255) / 256, tiles_n = (a.N + kPairN - 1) / kPairN;
  const int tiles = tiles_m * tiles_n;
  const int pair = blockIdx.x / (2 * SPLITS), pairs = gridDim.x / (2 * SPLITS);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairStages; ++s) mbar_init(&full[s], 1), mbar_init(&empty[s], 2);
    for (int b = 0; b < 4; ++b) mbar_init(&pfull[b], 1), mbar_init(&pempty[b], 8);
    mbar_init(&drain[0], 1), mbar_init(&drain[1], 1);
    *abort_flag = 0;
    fence_mbar_init_cluster();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  if (a.clear && blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;

  if (warp < 4) {
    regs_fewer<kPairFewRegs>();
    if (warp == 0) {
      // ---------------- TMA producer (both CTAs; the bytes complete on the leader's barrier).  Half h
      // of the tile's columns is rows 64 h .. 64 h + 63 of both CTAs' B.
      if (elect_one()) {
        tma_prefetch_desc(&tm_a);
        tma_prefetch_desc(&tm_b);
      }
      const uint32_t full_leader = mapa_shared(smem_addr(full), lead);
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued = 0, parities = 0;  // bit s: stage s was filled, and with which parity last
      bool ok = true;
      for (int tile = pair; ok && tile < tiles; tile += pairs) {
        const int m0 = (tile % tiles_m) * 256 + static_cast<int>(rank) * 128;
        const int n0 = (tile / tiles_m) * kPairN + static_cast<int>(rank) * 64;
        for (int kb = 0; kb < num_kb; ++kb) {
          ok = warp_wait(&empty[stage], phase ^ 1, abort_flag, a.status);
          if (!ok) break;
          uint8_t* st = smem + stage * kPairStageBytes;
          const uint32_t bar = full_leader + static_cast<uint32_t>(stage * sizeof(uint64_t));
          if (elect_one()) {
            if (leader) mbar_arrive_expect_tx(&full[stage], 2 * kPairStageBytes);
            tma_load_2d_pair(st, &tm_a, bar, (kb0 + kb) * kSlice, m0);
            tma_load_2d_pair(st + kSlice * kSlice, &tm_b, bar, (kb0 + kb) * kSlice, n0);
            tma_load_2d_pair(st + kSlice * kSlice + 64 * kSlice, &tm_b, bar, (kb0 + kb) * kSlice, n0 + 128);
          }
          __syncwarp();
          issued |= 1u << stage;
          parities = (parities & ~(1u << stage)) | (phase << stage);
          if (++stage == kPairStages) stage = 0, phase ^= 1;
        }
      }
      if (*abort_flag && leader) {
        // a bounded chance for the copies already issued to land before the pair exits
        int never = 0;
        for (int s = 0; s < kPairStages; ++s)
          if (issued >> s & 1) mbar_wait(&full[s], parities >> s & 1, &never, a.status, 0);
      }
    } else if ((warp == 1 || warp == 2) && leader) {
      // ---------------- MMA issuers: slice `it` of this pair's walk into TMEM buffer it & 1, warp 1 + h
      // for half h of the columns
      const uint32_t h = static_cast<uint32_t>(warp - 1);
      int stage = 0;
      uint32_t phase = 0;
      uint32_t it = 0;
      bool ok = true;
      for (int tile = pair; ok && tile < tiles; tile += pairs) {
        for (int kb = 0; kb < num_kb; ++kb, ++it) {
          const uint32_t b = it & 1;
          ok = warp_wait(&full[stage], phase, abort_flag, a.status) &&
               warp_wait(&pempty[2 * b + h], ((it >> 1) & 1) ^ 1, abort_flag, a.status);
          if (!ok) break;
          tc_fence_after();
          // a descriptor's address field counts 16 bytes: a K step is 2
          const uint64_t da = sdesc_kmajor_sw128(smem_addr(smem + stage * kPairStageBytes));
          const uint64_t db = sdesc_kmajor_sw128(smem_addr(smem + stage * kPairStageBytes + kSlice * kSlice + h * 64 * kSlice));
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc_mma_pair<kKindF8>(tmem + b * 256u + h * 128u, da + 2 * k, db + 2 * k, kIdesc, k > 0 ? 1u : 0u);
            tc_commit_pair_mc(&pfull[2 * b + h], both);
            tc_commit_pair_mc(&empty[stage], both);
          }
          __syncwarp();
          if (++stage == kPairStages) stage = 0, phase ^= 1;
        }
      }
      if (*abort_flag) {
        int never = 0;
        if (elect_one()) tc_commit_pair(&drain[h]);
        __syncwarp();
        mbar_wait(&drain[h], 0, &never, a.status, 0);
      }
    }
    if constexpr (SPLITS > 1) {  // the promotion warps' two cluster barriers
      __syncwarp();
      cluster_sync();
      cluster_sync();
    }
  } else {
    regs_more<kPairManyRegs>();
    // ---------------- promotion: warp w reads TMEM lanes 32 (w % 4) .. (its row) and the 128 columns of
    // half h of each buffer, h its warpgroup
    const int quarter = warp & 3, h = (warp - 4) >> 2;
    const int row = quarter * 32 + lane;
    const uint32_t pempty_leader = mapa_shared(smem_addr(&pempty[h]), lead);
    const uint32_t t_base = tmem + static_cast<uint32_t>(h * 128) + (static_cast<uint32_t>(quarter * 32) << 16);
    float* my_ring = rings + (warp - 4) * kRing * kRingFloats;
    const uint32_t ring = smem_addr(my_ring);
    uint32_t it = 0;
    bool ok = true;
    // The scales of a slice come through this warp's ring of kRing slots in shared memory, copied kRing - 1 slices
    // ahead, over the end of a tile into the next: lane l's row scale, and its column scales (the tile's one scale,
    // or of columns l, l + 32, l + 64, l + 96).
    const int64_t b_step = ROW_B ? static_cast<int64_t>(a.N) : a.sb_k;
    const float *pa, *pb;
    int next_tile = pair, next_kb = 0, next_n;  // the slice that is copied next
    auto aim = [&]() {
      const int m = (next_tile % tiles_m) * 256 + static_cast<int>(rank) * 128 + row;
      next_n = (next_tile / tiles_m) * kPairN + h * 128;
      pa = a.sa + static_cast<int64_t>(kb0) * a.M + (m < a.M ? m : 0);
      pb = a.sb + kb0 * b_step + (ROW_B ? 0 : static_cast<int64_t>(next_n < a.N ? next_n >> 7 : 0) * a.sb_n);
    };
    auto fetch = [&](uint32_t slot_of) {
      if (next_tile < tiles) {
        const uint32_t slot = ring + ((slot_of % kRing) * kRingFloats + static_cast<uint32_t>(lane)) * 4u;
        copy_async4(slot, pa);
#pragma unroll
        for (int e = 0; e < (ROW_B ? 4 : 1); ++e) {
          const int n = ROW_B ? next_n + 32 * e + lane : 0;
          copy_async4(slot + 128u * (1 + e), pb + (n < a.N ? n : 0));
        }
        pa += a.M, pb += b_step;
        if (++next_kb == num_kb) {
          next_kb = 0, next_tile += pairs;
          aim();
        }
      }
      copy_async_commit();
    };
    aim();
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) fetch(i);
    for (int tile = pair; tile < tiles; tile += pairs) {
      const int m = (tile % tiles_m) * 256 + static_cast<int>(rank) * 128 + row;
      const int ng = (tile / tiles_m) * kPairN + h * 128;
      const bool row_ok = m < a.M;
      float acc[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i] = 0.f;
      auto factor = [&]() {  // of this lane's row and the tile (with row scales: the reciprocals stay in the ring)
        copy_async_wait<kRing - 2>();
        float* v = my_ring + (it % kRing) * kRingFloats;
        if constexpr (ROW_B) {
#pragma unroll
          for (int e = 0; e < 5; ++e) v[32 * e + lane] = fast_rcp(v[32 * e + lane]);
          __syncwarp();
          return 0.f;
        }
        return fast_rcp(v[lane]) * fast_rcp(v[32 + lane]);
      };
      for (int kb = 0; kb < num_kb; ++kb, ++it) {
        const uint32_t b = it & 1;
        if (ok) ok = warp_wait(&pfull[2 * b + h], (it >> 1) & 1, abort_flag, a.status);
        if (!ok) continue;
        tc_fence_after();
        const uint32_t t = t_base + b * 256u;
        // the half buffer's columns in two loads of 64 (with row scales: of 16 lanes each, so that a thread holds
        // two columns of four rows and reads a quarter of the column factors), the next pair of loads on their way
        // while the first is added
        auto load = [&](int k, uint32_t(&p)[32]) {
          if constexpr (ROW_B)
            tmem_ld16x64(t + static_cast<uint32_t>((k >> 1) * 64) + (static_cast<uint32_t>((k & 1) * 16) << 16), p);
          else
            tmem_ld32(t + static_cast<uint32_t>(k * 32), p);
        };
        uint32_t p0[32], p1[32];
        load(0, p0);
        load(1, p1);
        const float f = factor();  // while the loads are on their way
        const float* fac = my_ring + (it % kRing) * kRingFloats;
        float2 cf[8];
        auto columns = [&](int c) {  // the factors of the thread's columns of load pair c
          if constexpr (ROW_B) {
#pragma unroll
            for (int i = 0; i < 8; ++i) cf[i] = *reinterpret_cast<const float2*>(fac + 32 + c * 64 + 8 * i + 2 * (lane & 3));
          }
        };
        auto add = [&](int k, const uint32_t(&p)[32]) {
          if constexpr (ROW_B) {
            const float lo = fac[(k & 1) * 16 + (lane >> 2)], hi = fac[(k & 1) * 16 + (lane >> 2) + 8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float w[4] = {cf[i].x * lo, cf[i].y * lo, cf[i].x * hi, cf[i].y * hi};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                acc[k * 32 + 4 * i + e] = fmaf(__uint_as_float(p[4 * i + e]), w[e], acc[k * 32 + 4 * i + e]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[k * 32 + i] = fmaf(__uint_as_float(p[i]), f, acc[k * 32 + i]);
          }
        };
        columns(0);
        tmem_ld_deps64(p0, p1);
        add(0, p0);
        load(2, p0);
        add(1, p1);
        load(3, p1);
        columns(1);
        tmem_ld_deps64(p0, p1);
        // this warp has read its part of the half buffer
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote_relaxed(pempty_leader + b * 2 * static_cast<uint32_t>(sizeof(uint64_t)));
        add(2, p0);
        add(3, p1);
        fetch(it + kRing - 1);
      }
      TO* dst = static_cast<TO*>(a.out) + static_cast<int64_t>(m) * a.N;
      if constexpr (SPLITS > 1) {
        // The pairs' partial sums meet in the CTAs' stage rings, once both pairs are done with their own: pair q
        // adds up half q of the tile's columns, in pair order.  (A cluster that splits K has one tile.)  Layout
        // [pair][column / 4][row][4], or with row scales, whose threads hold two columns of four rows,
        // [pair][column / 2][row ^ 8 (column / 2 % 4)][2].
        cluster_sync();
        const uint32_t owner = mapa_shared(smem_addr(smem) + static_cast<uint32_t>(part * 65536), static_cast<uint32_t>(2 * h) + rank);
        if constexpr (ROW_B) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              const int col2 = (k >> 1) * 32 + 4 * (j >> 2) + (lane & 3);
              const int r = quarter * 32 + (k & 1) * 16 + (j & 2) * 4 + (lane >> 2);
              asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(owner + col2 * 1024 + ((r ^ (8 * (lane & 3))) * 8)),
                           "f"(acc[k * 32 + j]), "f"(acc[k * 32 + j + 1])
                           : "memory");
            }
        } else {
#pragma unroll
          for (int j = 0; j < 128; j += 4)
            asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(owner + row * 16 + j * 512u), "f"(acc[j]), "f"(acc[j + 1]),
                         "f"(acc[j + 2]), "f"(acc[j + 3])
                         : "memory");
        }
        cluster_sync();
#pragma unroll 1
        for (int c = h * 64; c < h * 64 + 64; c += 32) {  // this warpgroup's half of the pair's columns
          float v[32];
          if constexpr (ROW_B) {
            const float2* in = reinterpret_cast<const float2*>(smem);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int at = (c / 2 + i) * 128 + (row ^ (8 * (i & 3)));
              const float2 t = in[at], w = in[8192 + at];
              v[2 * i] = t.x + w.x, v[2 * i + 1] = t.y + w.y;
            }
          } else {
            const float4* in = reinterpret_cast<const float4*>(smem) + row;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 t = in[(c / 4 + i) * 128], w = in[4096 + (c / 4 + i) * 128];
              v[4 * i] = t.x + w.x, v[4 * i + 1] = t.y + w.y, v[4 * i + 2] = t.z + w.z, v[4 * i + 3] = t.w + w.w;
            }
          }
          const int n = (tile / tiles_m) * kPairN + part * 128 + c;
          if (ok && row_ok && n < a.N) store_row<TO>(dst, a.bias, n, a.N, v);
        }
      } else if (ok) {
        // the warp's 32 x 128 outputs leave through two boxes in shared memory, which TMA stores while the warp
        // goes on (a thread's own 16-byte stores, a row each, take 2 us a tile)
        constexpr int kCols = 128 / static_cast<int>(sizeof(TO));  // columns of a box
        uint8_t* my_boxes = boxes + (warp - 4) * 2 * kBox;
#pragma unroll
        for (int x = 0; x < 128 / kCols; ++x) {
          uint8_t* box = my_boxes + (x & 1) * kBox;
          if (lane == 0) store_wait_read<1>();  // the box's last contents are read
          __syncwarp();
          if constexpr (ROW_B) {
            static_assert(sizeof(TO) == 4, "row scales have float32 outputs, and no bias");
#pragma unroll
            for (int i = 0; i < 16; ++i) {  // (half of the lanes, row + 8, group of 8 columns)
              const int k = (x >> 1) * 2 + (i >> 3), j = 16 * (x & 1) + 4 * (i & 3) + 2 * ((i >> 2) & 1);
              const int r = (i >> 3) * 16 + ((i >> 2) & 1) * 8 + (lane >> 2), q = lane & 3;
              *reinterpret_cast<float2*>(box + r * 128 + (((2 * (i & 3) + (q >> 1)) ^ (r & 7)) * 16) + (q & 1) * 8) =
                  make_float2(acc[k * 32 + j], acc[k * 32 + j + 1]);
            }
          } else {
#pragma unroll
            for (int c = 0; c < kCols / 8; ++c) {
              const int n = ng + x * kCols + c * 8;
              float v[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = acc[x * kCols + c * 8 + e];
              if (a.bias && n < a.N) {  // N is a multiple of 8
                const uint4 u = __ldg(reinterpret_cast<const uint4*>(a.bias + n));
                v[0] += bf16_lo(u.x), v[1] += bf16_hi(u.x), v[2] += bf16_lo(u.y), v[3] += bf16_hi(u.y);
                v[4] += bf16_lo(u.z), v[5] += bf16_hi(u.z), v[6] += bf16_lo(u.w), v[7] += bf16_hi(u.w);
              }
              if constexpr (sizeof(TO) == 2) {
                *reinterpret_cast<uint4*>(box + lane * 128 + ((c ^ (lane & 7)) * 16)) =
                    make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
              } else {
                *reinterpret_cast<float4*>(box + lane * 128 + (((2 * c) ^ (lane & 7)) * 16)) = make_float4(v[0], v[1], v[2], v[3]);
                *reinterpret_cast<float4*>(box + lane * 128 + (((2 * c + 1) ^ (lane & 7)) * 16)) = make_float4(v[4], v[5], v[6], v[7]);
              }
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (m < a.M && ng + x * kCols < a.N) tma_store_2d(&tm_out, box, ng + x * kCols, m);  // TMA clips the edges
            store_commit();
          }
        }
      }
    }
    if (SPLITS == 1 && lane == 0) store_wait<0>();
  }

  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ----------------------------------------------------------------------------- few rows
template <int NT>
struct StreamCfg {
  static constexpr int kStageBytes = kSlice * kSlice + NT * kSlice;
  static constexpr int kJoinBytes = NT * 128 * 4;               // the partial sums of this CTA's columns
  static constexpr int kStages = (104 * 1024 - kJoinBytes) / kStageBytes;  // two CTAs to an SM
  static constexpr int kBufs = 4;                               // slices' products in TMEM
  static constexpr int kTmemCols = kBufs * NT;
  static constexpr int kFacSlices = 8;                          // slices whose factors are held at a time
  static constexpr int kSmem = kStages * kStageBytes + kJoinBytes + 2 * kFacSlices * NT * 4 + 256 + 1024;
  static_assert(NT == 32 || NT == 64, "columns of a tile");
};
constexpr int kStreamThreads = 64 + 128;

template <int NT, bool ROW_B, typename TO>
__global__ void __launch_bounds__(kStreamThreads)
    block_stream_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                        const __grid_constant__ BlockArgs a) {
  using Cfg = StreamCfg<NT>;
  constexpr uint32_t kIdesc = make_idesc<kKindF8>(128, NT);
  constexpr int kFac = Cfg::kFacSlices;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* join = smem + Cfg::kStages * Cfg::kStageBytes;
  float* fac = reinterpret_cast<float*>(join + Cfg::kJoinBytes);  // [2][kFac][NT]
  uint64_t* full = reinterpret_cast<uint64_t*>(fac + 2 * kFac * NT);
  uint64_t* empty = full + Cfg::kStages;
  uint64_t* pfull = empty + Cfg::kStages;
  uint64_t* pempty = pfull + Cfg::kBufs;
  uint64_t* drain = pempty + Cfg::kBufs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = gridDim.x, rank = blockIdx.x;  // the cluster spans gridDim.x
  const int n0 = blockIdx.y * 128, m0 = blockIdx.z * NT;
  // this CTA's slices
  const int per = a.num_kb / splits, rest = a.num_kb - per * splits;
  const int kb0 = rank * per + (rank < rest ? rank : rest);
  const int num = per + (rank < rest ? 1 : 0);

  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::kStages; ++s) mbar_init(&full[s], 1), mbar_init(&empty[s], 1);
    for (int b = 0; b < Cfg::kBufs; ++b) mbar_init(&pfull[b], 1), mbar_init(&pempty[b], 4);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, Cfg::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (splits > 1) cluster_arrive();  // this CTA runs: its shared memory may be written
  pdl_wait();
  pdl_trigger();
  if (a.clear && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) *a.status = 0;

  auto wait = [&](uint64_t* bar, uint32_t parity) { return warp_wait(bar, parity, abort_flag, a.status); };
  float acc[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i] = 0.f;
  bool ok = true;

  if (warp == 0) {
    // ---------------- TMA producer
    if (elect_one()) {
      tma_prefetch_desc(&tm_a);
      tma_prefetch_desc(&tm_b);
    }
    int issued = 0, s = 0;
    uint32_t phase = 0;
    for (int i = 0; i < num; ++i) {
      if (!wait(&empty[s], phase ^ 1u)) break;
      uint8_t* st = smem + s * Cfg::kStageBytes;
      if (elect_one()) {
        mbar_arrive_expect_tx(&full[s], Cfg::kStageBytes);
        tma_load_2d(st, &tm_b, &full[s], (kb0 + i) * kSlice, n0);
        tma_load_2d(st + kSlice * kSlice, &tm_a, &full[s], (kb0 + i) * kSlice, m0);
      }
      __syncwarp();
      issued = i + 1;
      if (++s == Cfg::kStages) s = 0, phase ^= 1u;
    }
    if (*abort_flag) {
      int never = 0;
      for (int t = issued - Cfg::kStages > 0 ? issued - Cfg::kStages : 0; t < issued; ++t)
        mbar_wait(&full[t % Cfg::kStages], static_cast<uint32_t>(t / Cfg::kStages) & 1u, &never, a.status, 0);
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer: slice i into TMEM buffer i % kBufs
    int s = 0;
    uint32_t phase = 0;
    for (int i = 0; i < num; ++i) {
      const int b = i % Cfg::kBufs;
      if (!wait(&full[s], phase)) break;
      if (!wait(&pempty[b], (static_cast<uint32_t>(i / Cfg::kBufs) & 1u) ^ 1u)) break;
      tc_fence_after();
      const uint64_t dw = sdesc_kmajor_sw128(smem_addr(smem + s * Cfg::kStageBytes));
      const uint64_t dx = sdesc_kmajor_sw128(smem_addr(smem + s * Cfg::kStageBytes + kSlice * kSlice));
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc_mma<kKindF8>(tmem + static_cast<uint32_t>(b * NT), dw + 2 * k, dx + 2 * k, kIdesc, k > 0 ? 1u : 0u);
        tc_commit(&empty[s]);
        tc_commit(&pfull[b]);
      }
      __syncwarp();
      if (++s == Cfg::kStages) s = 0, phase ^= 1u;
    }
    if (*abort_flag) {
      int never = 0;
      if (elect_one()) tc_commit(drain);
      __syncwarp();
      mbar_wait(drain, 0, &never, a.status, 0);
    }
  } else {
    // ---------------- promotion: thread = one row of B, NT columns (rows of A)
    const int quarter = warp & 3, row = quarter * 32 + lane, tp = static_cast<int>(threadIdx.x) - 64;
    const uint32_t t_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    // factors of kFac slices at a time: entry (slice, column) by thread (slice * NT + column) % 128
    constexpr int kPer = kFac * NT / 128;
    float next[kPer];
    auto fetch = [&](int i0) {
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const int e = tp + u * 128, i = i0 + e / NT, m = m0 + e % NT;
        next[u] = 1.f;
        if (i < num && m < a.M) {
          next[u] = fast_rcp(__ldg(a.sa + static_cast<int64_t>(kb0 + i) * a.M + m));
          if constexpr (!ROW_B) next[u] *= fast_rcp(__ldg(a.sb + static_cast<int64_t>(blockIdx.y) * a.sb_n + (kb0 + i) * a.sb_k));
        }
      }
    };
    fetch(0);
    float sb_next = 1.f;
    const bool n_ok = n0 + row < a.N;
    if constexpr (ROW_B)
      if (n_ok && num > 0) sb_next = __ldg(a.sb + static_cast<int64_t>(kb0) * a.N + n0 + row);
    for (int i = 0; i < num; ++i) {
      const int b = i % Cfg::kBufs, slot = i % kFac, buf = (i / kFac) & 1;
      if (slot == 0) {
#pragma unroll
        for (int u = 0; u < kPer; ++u) fac[buf * kFac * NT + tp + u * 128] = next[u];
        fetch(i + kFac);
        asm volatile("bar.sync 1, 128;" ::: "memory");
      }
      float fr = 1.f;
      if constexpr (ROW_B) {
        fr = fast_rcp(sb_next);
        if (n_ok && i + 1 < num) sb_next = __ldg(a.sb + static_cast<int64_t>(kb0 + i + 1) * a.N + n0 + row);
      }
      if (ok) ok = wait(&pfull[b], static_cast<uint32_t>(i / Cfg::kBufs) & 1u);
      if (!ok) continue;
      tc_fence_after();
      const float* f = fac + (buf * kFac + slot) * NT;
      const uint32_t t = t_base + static_cast<uint32_t>(b * NT);
      auto add = [&](int c, const auto& p) {
#pragma unroll
        for (int q = 0; q < static_cast<int>(sizeof(p) / 16); ++q) {
          const float4 w = *reinterpret_cast<const float4*>(f + c + 4 * q);
          const float w4[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[c + 4 * q + e] = fmaf(__uint_as_float(p[4 * q + e]), ROW_B ? w4[e] * fr : w4[e], acc[c + 4 * q + e]);
        }
      };
      auto release = [&]() {  // this warp has read the buffer
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pempty[b]);
      };
      if constexpr (NT == 32) {
        uint32_t p[32];
        tmem_ld32_wait(t, p);
        release();
        add(0, p);
      } else {
        uint32_t p0[32], p1[32];
        tmem_ld64_wait(t, p0, p1);
        release();
        add(0, p0);
        add(32, p1);
      }
    }
  }

  auto put = [&](int m, int n, float v) {
    if (m >= a.M || n >= a.N) return;
    if (a.bias) v += __bfloat162float(a.bias[n]);
    TO* dst = static_cast<TO*>(a.out) + static_cast<int64_t>(m) * a.N + n;
    if constexpr (sizeof(TO) == 2)
      *dst = __float2bfloat16(v);
    else
      *dst = v;
  };
  const int row = (warp & 3) * 32 + lane;
  if (splits == 1) {
    if (warp >= 2 && ok) {
#pragma unroll
      for (int t = 0; t < NT; ++t) put(m0 + t, n0 + row, acc[t]);
    }
  } else {
    // CTA q of the cluster adds up columns [q cols, (q + 1) cols) of every CTA's partial sums, which the others
    // write into its join buffer as soon as they have them: [rank][cols / 4][row][4], so that a warp's 16-byte
    // stores and loads are contiguous
    const int shift = __ffs(NT / splits) - 1, cols = 1 << shift;
    __syncwarp();
    cluster_wait();  // every CTA of the cluster has started
    if (warp >= 2) {
      const uint32_t base = smem_addr(join) + static_cast<uint32_t>((rank << shift) * 512 + row * 16);
#pragma unroll
      for (int t = 0; t < NT; t += 4) {
        const uint32_t dst = mapa_shared(base + static_cast<uint32_t>((t & (cols - 1)) * 512), static_cast<uint32_t>(t >> shift));
        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "f"(acc[t]), "f"(acc[t + 1]),
                     "f"(acc[t + 2]), "f"(acc[t + 3])
                     : "memory");
      }
    }
    cluster_sync();
    if (warp >= 2 && ok) {
      const float4* part = reinterpret_cast<const float4*>(join) + row;
      for (int c = 0; c < cols; c += 4) {
        float4 w[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r < splits) w[r] = part[((r << shift) + c) * 32];
        float4 v = w[0];
#pragma unroll
        for (int r = 1; r < 8; ++r)
          if (r < splits) v.x += w[r].x, v.y += w[r].y, v.z += w[r].z, v.w += w[r].w;
        const int m = m0 + (rank << shift) + c;
        put(m, n0 + row, v.x), put(m + 1, n0 + row, v.y), put(m + 2, n0 + row, v.z), put(m + 3, n0 + row, v.w);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::kTmemCols);
  }
}

// ----------------------------------------------------------------------------- a few rows
// D (16 x 8, float32) += A (16 x 32) B (8 x 32)^T of E4M3 codes held in registers.
__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A CTA computes 16 rows of B against up to 8 CT rows of A; its 8 warps take the slices of K in turn.  Lane
// (g, q) = (lane / 4, lane % 4) of a warp copies 16 bytes at byte 16 q of both 64-byte halves of a slice, of
// rows g and g + 8 of B and of rows g, g + 8, .. of A: the four words of a copy are the lane's fragments of two
// MMAs, whose order along K is the same for both operands and otherwise free.  The copies land in a ring of
// kStages slices per warp in shared memory, in the lane's own places: no lane reads another's, so the ring
// needs no barrier, and every warp has kStages - 1 slices on their way while it works on one.  Three CTAs to
// an SM (72 or 64 KB) measured best: at 1 x 12288 x 4096 three stages take 11.2 us, two 11.2, four 13.4; at 16
// rows (CT = 2) two take 14.3, three 16.0.  D holds
// rows g, g + 8 and columns 2 q, 2 q + 1.
constexpr int kFewWarps = 8;
constexpr int kFewMaxSlices = 256;  // the factors 1 / (s_a s_b) of all slices are formed once, in shared memory
template <int CT>
struct FewCfg {
  static constexpr int kStages = CT == 1 ? 3 : 2;
  static constexpr int kStageBytes = (4 + 2 * CT) * 512;  // 16-byte pieces of 32 lanes
  static constexpr int kRingBytes = kFewWarps * kStages * kStageBytes;
  static int smem(int num_kb) { return kRingBytes + num_kb * 8 * CT * 4; }
};

template <int CT, typename TO>
__global__ void __launch_bounds__(32 * kFewWarps) block_few_kernel(const uint8_t* __restrict__ A, const uint8_t* __restrict__ B,
                                                                    int K, const BlockArgs a) {
  using Cfg = FewCfg<CT>;
  constexpr int kOut = 16 * 8 * CT;
  extern __shared__ __align__(128) uint8_t few_smem[];
  float* fac = reinterpret_cast<float*>(few_smem + Cfg::kRingBytes);  // [num_kb][8 CT]
  static_assert(kFewWarps * kOut * 4 <= Cfg::kRingBytes, "the partial sums reuse the ring");
  pdl_wait();
  pdl_trigger();
  if (a.clear && blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int n0 = blockIdx.x * 16;
  const uint32_t ring = smem_addr(few_smem) + static_cast<uint32_t>(warp * Cfg::kStages * Cfg::kStageBytes + lane * 16);
  const uint8_t* pb = B + static_cast<int64_t>(n0 + g) * K + 16 * q;
  const uint8_t* pa = A + static_cast<int64_t>(g) * K + 16 * q;
  const bool hi_ok = n0 + 8 < a.N;  // N is a multiple of 8: rows g are there
  const int64_t row8 = static_cast<int64_t>(8) * K;
  auto fetch = [&](int i) {  // this warp's i-th slice
    const int kb = warp + i * kFewWarps;
    if (kb < a.num_kb) {
      const uint32_t dst = ring + static_cast<uint32_t>((i % Cfg::kStages) * Cfg::kStageBytes);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = kb * kSlice + 64 * h;
        const bool ok = at + 16 * q < K;  // K is a multiple of 16
        copy_async16(dst + h * 512u, ok ? pb + at : B, ok);
        copy_async16(dst + (2 + h) * 512u, ok && hi_ok ? pb + row8 + at : B, ok && hi_ok);
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          const bool m_ok = ok && 8 * c + g < a.M;
          copy_async16(dst + (4 + 2 * c + h) * 512u, m_ok ? pa + c * row8 + at : A, m_ok);
        }
      }
    }
    copy_async_commit();
  };
#pragma unroll
  for (int i = 0; i < Cfg::kStages - 1; ++i) fetch(i);
  const float* sb = a.sb + static_cast<int64_t>(n0 >> 7) * a.sb_n;  // the rows of a CTA lie in one tile
  for (int i = threadIdx.x; i < a.num_kb * 8 * CT; i += 32 * kFewWarps) {
    const int kb = i / (8 * CT), m = i % (8 * CT);
    fac[i] = m < a.M ? fast_rcp(__ldg(a.sa + static_cast<int64_t>(kb) * a.M + m)) * fast_rcp(__ldg(sb + kb * a.sb_k)) : 0.f;
  }
  __syncthreads();
  float acc[CT][4];
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[c][e] = 0.f;
  for (int i = 0, kb = warp; kb < a.num_kb; ++i, kb += kFewWarps) {
    fetch(i + Cfg::kStages - 1);
    copy_async_wait<Cfg::kStages - 1>();
    const uint8_t* st = few_smem + (warp * Cfg::kStages + i % Cfg::kStages) * Cfg::kStageBytes + lane * 16;
    uint4 w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const uint4*>(st + j * 512);
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 x = *reinterpret_cast<const uint4*>(st + (4 + 2 * c + h) * 512);
        mma_e4m3(d, w[h].x, w[2 + h].x, w[h].y, w[2 + h].y, x.x, x.y);
        mma_e4m3(d, w[h].z, w[2 + h].z, w[h].w, w[2 + h].w, x.z, x.w);
      }
      const float2 f = *reinterpret_cast<const float2*>(fac + (kb * CT + c) * 8 + 2 * q);
      acc[c][0] = fmaf(d[0], f.x, acc[c][0]), acc[c][1] = fmaf(d[1], f.y, acc[c][1]);
      acc[c][2] = fmaf(d[2], f.x, acc[c][2]), acc[c][3] = fmaf(d[3], f.y, acc[c][3]);
    }
  }
  // the warps' sums, added in warp order; entry (column, row)
  copy_async_wait<0>();
  __syncthreads();
  float* red = reinterpret_cast<float*>(few_smem);
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[warp * kOut + (8 * c + 2 * q + (e & 1)) * 16 + g + 8 * (e >> 1)] = acc[c][e];
  __syncthreads();
  for (int i = threadIdx.x; i < kOut; i += 32 * kFewWarps) {
    const int m = i / 16, n = n0 + i % 16;
    if (m >= a.M || n >= a.N) continue;
    float v = 0.f;
#pragma unroll
    for (int s = 0; s < kFewWarps; ++s) v += red[s * kOut + i];
    if (a.bias) v += __bfloat162float(a.bias[n]);
    TO* dst = static_cast<TO*>(a.out) + static_cast<int64_t>(m) * a.N + n;
    if constexpr (sizeof(TO) == 2)
      *dst = __float2bfloat16(v);
    else
      *dst = v;
  }
}

// ----------------------------------------------------------------------------- host
// Whether a kernel's dynamic shared memory size has been set on a device (one flag per kernel and device).
struct Configured {
  std::atomic<uint64_t> devices{0};
};

template <typename F>
cudaError_t configure(F kern, int smem, Configured& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.devices.load(std::memory_order_acquire) & bit) return cudaSuccess;
  if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
  done.devices.fetch_or(bit, std::memory_order_release);
  return cudaSuccess;
}

bool code_map(CUtensorMap* map, const void* base, int64_t rows, int64_t k, int64_t ld, int box_rows) {
  const uint64_t dims[2] = {static_cast<uint64_t>(k), static_cast<uint64_t>(rows)};
  const uint64_t stride[1] = {static_cast<uint64_t>(ld)};
  const uint32_t box[2] = {static_cast<uint32_t>(kSlice), static_cast<uint32_t>(box_rows)};
  return encode_tmap(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, stride, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <bool ROW_B, typename TO, int SPLITS>
cudaError_t run_pair(const BlockGemm& p, const BlockArgs& a, int64_t tiles, cudaStream_t stream) {
  CUtensorMap ta, tb, to;
  const uint64_t dims[2] = {static_cast<uint64_t>(p.N), static_cast<uint64_t>(p.M)}, stride[1] = {p.N * sizeof(TO)};
  const uint32_t box[2] = {static_cast<uint32_t>(128 / sizeof(TO)), 32};
  if (!code_map(&ta, p.A, p.M, p.K, p.lda, 128) || !code_map(&tb, p.B, p.N, p.K, p.ldb, 64) ||
      !encode_tmap(&to, sizeof(TO) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, p.out, dims,
                   stride, box, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  auto kern = block_pair_kernel<ROW_B, TO, SPLITS>;
  static Configured done;
  cudaError_t e = configure(kern, kPairSmem, done);
  if (e != cudaSuccess) return e;
  const int most = num_sms() / (2 * SPLITS);
  if (SPLITS > 1 && tiles > most) return cudaErrorInvalidValue;  // a cluster that splits K joins once
  const unsigned clusters = static_cast<unsigned>(tiles < most ? tiles : most);
  e = launch_pdl(kern, dim3(2 * SPLITS * clusters), dim3(kPairThreads), kPairSmem, stream, ta, tb, to, a);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

// How many clusters of four SMs the current device has room for at once (two pairs of CTAs, an SM each).  Fewer than its
// SMs make, because a cluster lies within a group of SMs whose number need not be a multiple of four (36 of 38 on
// 152 SMs).  Asked once per kernel and device.
template <bool ROW_B, typename TO>
cudaError_t four_sm_places(int* places) {
  static std::atomic<int> known[64];  // places + 1
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int had = known[dev & 63].load(std::memory_order_relaxed);
  if (had > 0) return *places = had - 1, cudaSuccess;
  auto kern = block_pair_kernel<ROW_B, TO, 2>;
  static Configured done;
  if ((e = configure(kern, kPairSmem, done)) != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 4, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(4), cfg.blockDim = dim3(kPairThreads), cfg.dynamicSmemBytes = kPairSmem;
  cfg.attrs = attr, cfg.numAttrs = 1;
  if ((e = cudaOccupancyMaxActiveClusters(places, kern, &cfg)) != cudaSuccess) return e;
  known[dev & 63].store(*places + 1, std::memory_order_relaxed);
  return cudaSuccess;
}

// launch_pdl with clusters of `cluster` CTAs along x.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kern)(KArgs...), dim3 grid, int cluster, int threads, int smem, cudaStream_t stream, Args... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster), attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_next_launch() ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

template <int NT, bool ROW_B, typename TO>
cudaError_t run_stream(const BlockGemm& p, const BlockArgs& a, int splits, cudaStream_t stream) {
  using Cfg = StreamCfg<NT>;
  CUtensorMap ta, tb;
  if (!code_map(&ta, p.A, p.M, p.K, p.lda, NT) || !code_map(&tb, p.B, p.N, p.K, p.ldb, 128)) return cudaErrorInvalidValue;
  auto kern = block_stream_kernel<NT, ROW_B, TO>;
  static Configured done;
  cudaError_t e = configure(kern, Cfg::kSmem, done);
  if (e != cudaSuccess) return e;
  return launch_cluster(kern, dim3(splits, (p.N + 127) / 128, (p.M + NT - 1) / NT), splits, kStreamThreads, Cfg::kSmem, stream,
                        ta, tb, a);
}

template <int CT, typename TO>
cudaError_t run_few(const BlockGemm& p, const BlockArgs& a, cudaStream_t stream) {
  auto kern = block_few_kernel<CT, TO>;
  static Configured done;
  cudaError_t e = configure(kern, FewCfg<CT>::smem(kFewMaxSlices), done);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3((p.N + 15) / 16), dim3(32 * kFewWarps), FewCfg<CT>::smem(a.num_kb), stream, p.A, p.B, p.K, a);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

// Which kernel, with both sides of each rule (GPU times from captured graphs, M x N x K).
// Up to 8 rows, or 16 with K up to 8192, the few-row kernel, as the weights' bytes and the launch are the cost: 1 x 6144
// x 4096 5.7 us against 8.1 in the stream kernel, 1 x 1024 x 1024 2.2 against 4.3, 8 x 4096 x 14336 14.6 against 14.4, 16 x
// 4096 x 4096 6.1 against 7.1, x 6144 8.0 against 7.9, x 8192 10.2 against 8.9, x 14336 18.2 against 14.4.  (With 9 to 16
// rows and more columns the border lies lower than the rule has it: 16 x 8192 x 4096 10.5 against 9.2, x 8192 20.1
// against 15.8.)
// From 65 rows on the pair kernel once its tiles take 2 of 5 pairs: 32 tiles, 512 x 4096 x 4096 16.6 us against 26.2, x
// 1024 9.9 against 10.4; tiles half empty, 128 x 7936 x 4096 16.9 against 18.3, 96 x 12288 x 4096 23.0 against 26.7; a
// quarter full, 64 x 12288 x 4096 22.8 against 19.1; fewer tiles, 128 x 6144 x 4096 (24) 16.1 against 17.0, 128 x 4096 x
// 4096 (16) 15.9 against 10.5.
// Two pairs to a tile from 16 slices on where all of them have a place at once: 512 x 4096 x 14336 36.7 us against 61.3 on
// one, x 2048 12.6 against 13.8, x 1536 (12 slices) 11.6 against 11.9, x 1024 10.6 against 9.9; 37 tiles on 36 places,
// 256 x 9472 x 2048, 22.5 against 13.8; four pairs, clusters of eight, left SMs idle.  It pays from 16 tiles on if none of
// them is half empty: 256 x 4096 x 14336 36.0 us against 43.6 in the stream kernel, x 4096 15.8 against 16.6; half empty,
// 128 x 4096 x 14336 35.9 against 25.7.
// With row scales (dW, times with the gradient's cast) the stream kernel comes nearer: 32 tiles of 2048 x 1024, 32 slices 29.5
// us against 33.4, 16 19.0 against 18.7, 8 15.1 against 12.6; 16 tiles of 1024 x 1024, 32 slices 25.1 against 19.7.
// Between them the stream kernel, K split while two CTAs to an SM still hold every CTA of the launch (64 x 4096 x 14336:
// 68.5, 38.0, 22.2, 17.8 us on 1, 2, 4, 8; 32 x 12288 x 4096, 96 tiles: 18.3, 14.5, 17.1 on 1, 2, 4), clusters of eight only
// while each has a place (64 x 4736 x 2048, 37 tiles on 36 places: 11.2 us, on clusters of four 7.7; x 14336 27.6 and
// 25.7).  Clusters of four had 74 places: with 75 and 76 tiles they take 13.2 us where two CTAs take 9.4, which
// nothing that can be asked of the device foretells.
template <bool ROW_B, typename TO>
cudaError_t run_any(const BlockGemm& p, const BlockArgs& a, cudaStream_t stream) {
  if constexpr (!ROW_B)
    if (p.M <= 16 && a.num_kb <= (p.M <= 8 ? kFewMaxSlices : 64) && p.lda == p.K && p.ldb == p.K)
      return p.M <= 8 ? run_few<1, TO>(p, a, stream) : run_few<2, TO>(p, a, stream);
  const int64_t pair_tiles = static_cast<int64_t>((p.M + 255) / 256) * ((p.N + kPairN - 1) / kPairN);
  if (pair_tiles > INT32_MAX) return cudaErrorInvalidValue;
  bool split = 4 * pair_tiles <= num_sms() && a.num_kb >= 16;
  if (split) {
    int places = 0;
    const cudaError_t e = four_sm_places<ROW_B, TO>(&places);
    if (e != cudaSuccess) return e;
    split = pair_tiles <= places;
  }
  if (p.M > 64 && (pair_tiles >= num_sms() / 5 || (split && p.M > 128 && pair_tiles >= num_sms() / 10)))
    return split ? run_pair<ROW_B, TO, 2>(p, a, pair_tiles, stream) : run_pair<ROW_B, TO, 1>(p, a, pair_tiles, stream);
  const int nt = p.M <= 32 ? 32 : 64;
  const int64_t tiles = static_cast<int64_t>((p.N + 127) / 128) * ((p.M + nt - 1) / nt);
  int splits = 1;
  while (splits < 8 && 2 * splits <= a.num_kb && tiles * 2 * splits <= 2 * num_sms()) splits *= 2;
  if (splits == 8) {  // eight CTAs, two to an SM
    int places = 0;
    const cudaError_t e = four_sm_places<ROW_B, TO>(&places);
    if (e != cudaSuccess) return e;
    if (tiles > places) splits = 4;
  }
  return nt == 32 ? run_stream<32, ROW_B, TO>(p, a, splits, stream) : run_stream<64, ROW_B, TO>(p, a, splits, stream);
}

}  // namespace

cudaError_t launch_gemm_block(const BlockGemm& p, uint32_t* status, int clear_status, cudaStream_t stream) {
  if (p.M <= 0 || p.N <= 0) return cudaSuccess;
  if (p.K <= 0) return cudaErrorInvalidValue;
  BlockArgs a;
  a.sa = p.sa, a.sb = p.sb, a.sb_n = p.sb_n, a.sb_k = p.sb_k;
  a.bias = p.bias, a.out = p.out, a.M = p.M, a.N = p.N, a.num_kb = (p.K + kSlice - 1) / kSlice;
  a.status = status, a.clear = clear_status;
  if (p.row_b) return p.out_f32 ? run_any<true, float>(p, a, stream) : cudaErrorInvalidValue;
  return p.out_f32 ? run_any<false, float>(p, a, stream) : run_any<false, __nv_bfloat16>(p, a, stream);
}

}  // namespace mmdit
