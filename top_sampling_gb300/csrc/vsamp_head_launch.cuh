// Launch of the 4-bit head: geometry and the instantiation for a number of column tiles and a group size. Each group
// size is a translation unit of its own, which defines VSAMP_HEAD_KERNELS (vsamp_head_g32.cu, vsamp_head_g64.cu, vsamp_head_g128.cu).
#pragma once

#include <atomic>

#include "vsamp_grid.h"
#include "vsamp_head.cuh"
#include "vsamp_host.h"

namespace vsamp {

template <int GROUP>
vsamp_status launch_head_group(const HeadParams& p, const DeviceInfo& d, int dev, cudaStream_t s);

#ifdef VSAMP_HEAD_KERNELS
template <int NT, int RT, int GROUP, int SB, bool ZEROS, int PF, int MAXW>
static vsamp_status launch_head_cfg(HeadParams p, const DeviceInfo& d, int dev, cudaStream_t stream) {
  auto kern = head_kernel<NT, RT, GROUP, SB, ZEROS, PF, MAXW>;
  const int64_t sets = (p.s.tiles() + RT - 1) / RT, sms = d.sm_count;
  // Warps per CTA: as many rounds over the row tiles as the largest CTA needs, each with as few warps as that allows,
  // so that the last round is nearly full. With fewer tiles than warps, warps share tiles along the inner dimension.
  const int64_t per_sm = (sets + sms - 1) / sms, rounds = (per_sm + MAXW - 1) / MAXW;
  int warps = (int)((per_sm + rounds - 1) / rounds);
  p.split = 1;
  if (rounds == 1) {
    while (sets * p.split * 2 <= sms * MAXW && p.split * 2 <= p.units && p.split < 8) p.split *= 2;
    warps = (int)((sets * p.split + sms - 1) / sms);
    warps = (warps + p.split - 1) / p.split * p.split;
  }
  const int red = p.split > 1 ? warps * RT * NT * 4 * 32 * 4 : 0;
  const int64_t unit_bytes = (int64_t)kHeadUnitSteps * NT * 8 * 32;
  const int ring = warps * PF * RT * p.s.record();
  const int64_t most = (d.optin - red - ring) / unit_bytes;
  if (most < 1) return VSAMP_ERR_UNSUPPORTED;
  p.chunk = p.units <= most ? p.units : (int)most;
  p.ring_off = (int)(p.chunk * unit_bytes);
  p.red_off = p.ring_off + ring;
  const int smem = p.red_off + red;
  // the kernel's limit is raised to the device's once, so concurrent callers never lower it under each other
  static std::atomic<bool> raised[64];
  if (dev >= 64 || !raised[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, d.optin) != cudaSuccess) {
      cudaGetLastError();
      return VSAMP_ERR_CUDA;
    }
    if (dev < 64) raised[dev].store(true, std::memory_order_release);
  }
  const int64_t ctas = (sets * p.split + warps - 1) / warps;
  return launch_1d(kern, grid_of(ctas < sms ? ctas : sms), (unsigned)warps * 32, (size_t)smem, stream, p);
}

template <int NT, int RT, int GROUP, int PF, int MAXW>
static vsamp_status launch_head_nt(const HeadParams& p, const DeviceInfo& d, int dev, cudaStream_t s) {
  if (p.s.scale_bytes == 4)
    return p.s.has_zeros ? launch_head_cfg<NT, RT, GROUP, 4, true, PF, MAXW>(p, d, dev, s)
                         : launch_head_cfg<NT, RT, GROUP, 4, false, PF, MAXW>(p, d, dev, s);
  return p.s.has_zeros ? launch_head_cfg<NT, RT, GROUP, 2, true, PF, MAXW>(p, d, dev, s)
                       : launch_head_cfg<NT, RT, GROUP, 2, false, PF, MAXW>(p, d, dev, s);
}

template <int GROUP>
vsamp_status launch_head_group(const HeadParams& p, const DeviceInfo& d, int dev, cudaStream_t s) {
  const int nt = p.terms * p.term_tiles;
  if (nt == 1) {
    // Four row tiles per warp share the staged states and hide each other's latency (151936 x 4096: 55 us against 62
    // with one); with fewer than about 12 tiles per SM one tile per warp spreads them over more SMs (1000 x 4096: 4.4
    // against 7.2 us, 16000 x 4096: 12.4 against 13.9, 32000 x 2048: 12.2 against 11.8).
    if (p.s.tiles() < 12 * (int64_t)d.sm_count) return launch_head_nt<1, 1, GROUP, 4, 16>(p, d, dev, s);
    return launch_head_nt<1, 4, GROUP, 2, 16>(p, d, dev, s);
  }
  if (nt == 2) return launch_head_nt<2, 2, GROUP, 2, 16>(p, d, dev, s);
  if (nt == 3) return launch_head_nt<3, 2, GROUP, 2, 16>(p, d, dev, s);
  if (nt == 4) return launch_head_nt<4, 2, GROUP, 2, 16>(p, d, dev, s);
  if (nt <= 6) return launch_head_nt<6, 1, GROUP, 2, 16>(p, d, dev, s);
  return launch_head_nt<8, 1, GROUP, 2, 16>(p, d, dev, s);
}
#endif   // VSAMP_HEAD_KERNELS

}  // namespace vsamp
