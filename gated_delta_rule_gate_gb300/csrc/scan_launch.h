// scan_launch.h -- host-side launchers of the gated linear recurrence (internal
// to libgdn).  `act` and `gate` are gdn_dtype values; gate is F32 or act.
#pragma once

#include "scan.cuh"

namespace gdn {
namespace scan {

cudaError_t launch_step(const Args &p, int act, int gate, bool vec4, cudaStream_t stream);
cudaError_t launch_scan(const Args &p, int act, int gate, cudaStream_t stream);
cudaError_t launch_grad(const GradArgs &p, int act, int gate, cudaStream_t stream);
// One activation type each, rows on 16-byte addresses (p.wide) or anywhere, so that
// they compile side by side.
cudaError_t launch_scan_f32(const Args &p, cudaStream_t stream);
cudaError_t launch_scan_f16(const Args &p, bool gate_f32, cudaStream_t stream);
cudaError_t launch_scan_bf16(const Args &p, bool gate_f32, cudaStream_t stream);
cudaError_t launch_scan_f32_loose(const Args &p, cudaStream_t stream);
cudaError_t launch_scan_f16_loose(const Args &p, bool gate_f32, cudaStream_t stream);
cudaError_t launch_scan_bf16_loose(const Args &p, bool gate_f32, cudaStream_t stream);
cudaError_t launch_grad_f32(const GradArgs &p, cudaStream_t stream);
cudaError_t launch_grad_f16(const GradArgs &p, bool gate_f32, cudaStream_t stream);
cudaError_t launch_grad_bf16(const GradArgs &p, bool gate_f32, cudaStream_t stream);
cudaError_t launch_grad_f32_loose(const GradArgs &p, cudaStream_t stream);
cudaError_t launch_grad_f16_loose(const GradArgs &p, bool gate_f32, cudaStream_t stream);
cudaError_t launch_grad_bf16_loose(const GradArgs &p, bool gate_f32, cudaStream_t stream);

}  // namespace scan
}  // namespace gdn
