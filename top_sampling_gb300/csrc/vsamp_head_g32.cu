#define VSAMP_HEAD_KERNELS
#include "vsamp_head_launch.cuh"

namespace vsamp {
template vsamp_status launch_head_group<32>(const HeadParams&, const DeviceInfo&, int, cudaStream_t);
}
