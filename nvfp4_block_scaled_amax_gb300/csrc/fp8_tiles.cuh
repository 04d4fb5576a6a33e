// fp8_tiles.cuh -- what the product kernels of block-scaled E4M3 operands
// share: the list of output tiles over all members, tensor-core and copy
// primitives, and the scaled accumulation.
#pragma once

#include "common.cuh"
#include "dependent.h"
#include "fp8.h"
#include "tokens.h"

namespace nvfp4 {
namespace fp8 {

constexpr int kBK = 128;  // elements (bytes) of a block along the contracted dimension

// Beside the bits of common.cuh in the status word: member offsets that the call does not take.
constexpr unsigned kStatusOffsets = 4u;

struct MatmulKernelArgs {
  const float* sa;
  const float* sb;
  int64_t a_rows, a_cols, b_rows;
  int experts, wgrad;
  const int32_t* offsets;
  void* out;
  int out_bf16, out_map;
  unsigned* status;
};

// ---------------------------------------------------------------------------
// Members and tiles
// ---------------------------------------------------------------------------
// Member e holds the rows (wgrad: columns) offsets[e] .. offsets[e + 1] of A.
// Member `experts` of a forward product is the rows past the last member:
// nothing to sum, zeros to write.
__device__ __forceinline__ int member_count(const MatmulKernelArgs& p) {
  return p.offsets == nullptr ? 1 : p.experts + (p.wgrad ? 0 : 1);
}

// One tile: rows a_row .. of A and b_row .. of B (coordinates of the tensor
// maps), blocks kb0 .. kb0 + nkb, its place in the output and how much of it
// exists.
struct Tile {
  int64_t a_row, b_row, n0, out_row;
  int rows, cols;
  int kb0, nkb;
  int member;
};

// Tiles of kTM rows of A by kTN rows of B, all members in one list, in shared
// memory: first[i] is the first tile of member i (first[members]: the number of
// tiles), and kept behind them where each member begins.  Inside a member, bands of kBand row tiles,
// and in a band all row tiles of a column before the next column, so that the
// tiles in flight share both operands' rows in L2.  kBand 0: one band.
template <int kTM, int kTN, int kBand>
struct TileList {
  // Integers for `experts` members.
  static constexpr __host__ __device__ int ints(int experts) { return 2 * experts + 3; }
  // One warp fills the list.  Offsets that are no valid ones are reported, and
  // made to cut A into members all the same (each at least the one before, none
  // outside A), so that whatever they are the tiles are counted, read and written
  // inside the tensors and no two members share a row of the output.
  static __device__ __forceinline__ void fill(const MatmulKernelArgs& p, int* first) {
    const int lane = threadIdx.x & 31, members = member_count(p);
    const int limit = (int)(p.wgrad ? p.a_cols : p.a_rows);
    int* start = first + members + 1;
    if (p.offsets != nullptr) {
      bool bad = false;
      for (int e = lane; e <= p.experts; e += 32) {
        const int v = p.offsets[e], before = e > 0 ? p.offsets[e - 1] : 0;
        bad |= v < before || v > limit;
        // rows before the first member would stay unwritten; a block of two members has one scale
        bad |= p.wgrad ? v % kBK != 0 && v != limit : e == 0 && v != 0;
        start[e] = max(0, min(v, limit));
      }
      __syncwarp();
      if (__any_sync(0xFFFFFFFFu, bad)) {
        if (lane == 0) {
          atomicOr(p.status, kStatusOffsets);
          for (int e = 1; e <= p.experts; ++e) start[e] = max(start[e], start[e - 1]);
        }
        __syncwarp();
      }
    }
    const int64_t tn = (p.b_rows + kTN - 1) / kTN;
    int run = 0;
    for (int e0 = 0; e0 < members; e0 += 32) {
      const int e = e0 + lane;
      int64_t rows = p.wgrad ? p.a_rows : limit;
      if (p.offsets != nullptr && !p.wgrad && e < members) rows = (e < p.experts ? start[e + 1] : limit) - start[e];
      const int tiles = e < members ? (int)((rows + kTM - 1) / kTM * tn) : 0;
      int incl = tiles;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += v;
      }
      if (e < members) first[e] = run + incl - tiles;
      run += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    if (lane == 0) first[members] = run;
  }
  static __device__ __forceinline__ Tile at(const MatmulKernelArgs& p, const int* first, int t) {
    int lo = 0, hi = member_count(p);
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= t) lo = mid; else hi = mid;
    }
    Tile r;
    r.member = lo;
    const int i = t - first[lo];
    int64_t begin = 0, end = p.wgrad ? p.a_cols : p.a_rows;
    if (p.offsets != nullptr) {
      const int* start = first + member_count(p) + 1;
      begin = start[lo];
      if (lo < p.experts) end = start[lo + 1];
    }
    const int64_t M = p.wgrad ? p.a_rows : end - begin;
    const int mt = (int)((M + kTM - 1) / kTM), nt = (int)((p.b_rows + kTN - 1) / kTN);
    const int band = kBand ? i / (kBand * nt) : 0, in_band = i - band * kBand * nt;
    const int height = kBand ? min(kBand, mt - band * kBand) : mt;
    const int column = height == 1 ? in_band : (int)((unsigned)in_band / (unsigned)height);
    const int64_t m0 = (int64_t)(band * kBand + in_band - column * height) * kTM;
    r.n0 = (int64_t)column * kTN;
    r.rows = (int)min((int64_t)kTM, M - m0);
    r.cols = (int)min((int64_t)kTN, p.b_rows - r.n0);
    if (p.wgrad) {
      r.a_row = m0;
      r.b_row = r.n0;
      r.out_row = lo * p.a_rows + m0;
      r.kb0 = (int)(begin / kBK);
      r.nkb = begin == end ? 0 : (int)((end + kBK - 1) / kBK) - r.kb0;
    } else {
      const bool past = lo == p.experts;
      r.a_row = r.out_row = begin + m0;
      r.b_row = past ? 0 : lo * p.b_rows + r.n0;
      r.kb0 = 0;
      r.nkb = past ? 0 : (int)((p.a_cols + kBK - 1) / kBK);
    }
    return r;
  }
};

// ---------------------------------------------------------------------------
// Copies, barriers, tensor cores
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int32_t c0, int32_t c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
// The same, completing on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, int32_t c0, int32_t c1,
                                              uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
// Waits for a phase of an mbarrier, with a limit: false when it has not come
// after 2^19 tries.  A try that fails lasts up to 2600 cycles (measured), so
// that is about 0.7 s.  Unlike the wait of common.cuh it gives no time hint (a
// hinted try sleeps, up to half a microsecond too long for hand-overs every
// 0.3 us) and is a few instructions, for loops that must stay small.
__device__ __forceinline__ bool mbar_wait_at(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .u32 n;\n mov.u32 n, 524288;\n"
      "W:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra D;\n"
      " sub.u32 n, n, 1;\n setp.ne.u32 q, n, 0;\n @q bra W;\n"
      "D:\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity) {
  return mbar_wait_at(smem_u32(bar), parity);
}
// One warp's role gave up waiting: for nvfp4_device_status.
__device__ __forceinline__ void report_timeout(unsigned* status) { atomicOr(status, kStatusWaitTimeout); }
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Arrive on a barrier of the cluster (an address from map_to_cta).  The
// arrival orders tensor-memory reads only (complete, and fenced with
// tcgen05.fence::before_thread_sync), so it needs no cluster-scope release: that
// waits for every outstanding memory operation of the thread, about 1 us.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// 2D tiled store of the box at (c0, c1) from shared memory, in this thread's
// bulk group; what lies outside the tensor is not written.
__device__ __forceinline__ void tma_store(const CUtensorMap* map, uint32_t src, int32_t c0, int32_t c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(src)
               : "memory");
}
// Four floats to the shared memory of a CTA of the cluster, their bytes counted
// on a barrier of that CTA (both addresses from map_to_cta): the owner hears
// of them without an arrival that would first wait for them.
__device__ __forceinline__ void store_async(uint32_t dst, float a, float b, float c, float d, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(dst),
               "f"(a), "f"(b), "f"(c), "f"(d), "r"(bar)
               : "memory");
}
// For the cluster's shared memory: an arrival after the thread's earlier
// accesses, and a wait that sees what was written before the phase ended.
__device__ __forceinline__ void mbar_arrive_cluster_release(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, unsigned* status) {
  const long long t0 = clock64();
  uint32_t ok = 0;
  while (!ok) {
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (!ok && clock64() - t0 > kWaitLimitCycles) {
      atomicOr(status, kStatusWaitTimeout);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ uint32_t map_to_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// The same without ordering memory (which waits for the thread's stores in flight).
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// Four bytes to shared memory, asynchronously; zeros when `there` is false.
__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}
// One of the barrier's expected arrivals when this thread's cp.async copies so far are done.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The warp's index as a value the compiler knows to be the same in all lanes:
// the roles' loops then run on the uniform datapath, which the tensor-core
// instructions take their operands from.
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0); }
// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}

// Instruction descriptor of kind::f8f6f4: E4M3 A and B, both K-major, FP32 D.
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
// Operand descriptor of a K-major tile of 128-byte rows in the 128-byte
// swizzle (8-row groups 1024 bytes apart).
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) { return umma_smem_desc(addr, 16, 1024, 2); }
template <int kGroup>
__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  if constexpr (kGroup == 2)
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
                 "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
                 : "memory");
  else
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
                 "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
                 : "memory");
}
// One arrival on the barrier at this offset in both CTAs of the pair when
// every MMA this thread issued so far is complete.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Whole warp: consecutive columns of the lane into registers, complete on
// return.  (The load and its wait are one statement: with loads in flight
// across statements the compiler kept moving their registers, and the sum
// loop ran at half its speed.)
__device__ __forceinline__ void tmem_read(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_read(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]),
        "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]),
        "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_read(uint32_t taddr, uint32_t (&v)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, "
      "%45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, "
      "%62, %63}, [%64];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]),
        "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]),
        "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31]), "=r"(v[32]), "=r"(v[33]), "=r"(v[34]),
        "=r"(v[35]), "=r"(v[36]), "=r"(v[37]), "=r"(v[38]), "=r"(v[39]), "=r"(v[40]), "=r"(v[41]),
        "=r"(v[42]), "=r"(v[43]), "=r"(v[44]), "=r"(v[45]), "=r"(v[46]), "=r"(v[47]), "=r"(v[48]),
        "=r"(v[49]), "=r"(v[50]), "=r"(v[51]), "=r"(v[52]), "=r"(v[53]), "=r"(v[54]), "=r"(v[55]),
        "=r"(v[56]), "=r"(v[57]), "=r"(v[58]), "=r"(v[59]), "=r"(v[60]), "=r"(v[61]), "=r"(v[62]),
        "=r"(v[63])
      : "r"(taddr)
      : "memory");
}
// Whole warp: 64 columns of its 32 lanes in the 16 x 256-bit shape, complete on
// return: u from lanes 0-15, v from lanes 16-31.  Registers 4 j .. 4 j + 3 of
// thread t are rows t / 4, t / 4, t / 4 + 8, t / 4 + 8 of the 16 and columns
// 8 j + 2 (t mod 4) + {0, 1, 0, 1}: four rows of few columns, where the 32 x 32-bit
// shape gives a thread one row of all of them.
__device__ __forceinline__ void tmem_read_16x256(uint32_t taddr, uint32_t (&u)[32], uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31}, [%64];\n"
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%32, %33, %34, %35, %36, %37, %38, %39, %40, "
      "%41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, "
      "%58, %59, %60, %61, %62, %63}, [%65];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
        "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
        "=r"(u[14]), "=r"(u[15]), "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]),
        "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]),
        "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31]), "=r"(v[0]), "=r"(v[1]), "=r"(v[2]),
        "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]),
        "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
        "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]),
        "=r"(v[31])
      : "r"(taddr), "r"(taddr + (16u << 16))
      : "memory");
}

// Whole warp: 16 consecutive columns of the lane from registers, complete on return.
__device__ __forceinline__ void tmem_write(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15};\n"
      "tcgen05.wait::st.sync.aligned;" ::"r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(taddr)
      : "memory");
}

// Two FP32 values in a 64-bit register pair, and arithmetic on both.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// fp8_matmul_thin.cu: how it would cut a product (rows of A per tile, tiles
// expected, CTAs that share a tile's blocks), and the product so cut.
struct ThinPlan {
  int bn, split;
  int64_t tiles;
};
ThinPlan thin_plan(const Fp8MatmulArgs& a, const LaunchCtx& ctx);
cudaError_t launch_matmul_thin(const Fp8MatmulArgs& a, const MatmulKernelArgs& p, const LaunchCtx& ctx);

}  // namespace fp8
}  // namespace nvfp4
