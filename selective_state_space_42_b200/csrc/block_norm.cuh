// block_norm.cuh -- launch parameters and entry points of the block-norm
// junction and its gradient (block_norm.cu).
#pragma once

#include "selscan_device.cuh"

namespace selscan {

constexpr int kBnMaxDim = 16384;
constexpr int kBnMaxGroups = 1024;
enum { kGateNone = 0, kGateBefore = 1, kGateAfter = 2 };

struct BlockNormParams {
    const void *x, *z;                  // rows of dim elements, x_row / z_row apart
    long long x_row, z_row;
    const float *weight, *res_scale, *next_weight;  // [dim] or NULL
    const void *res;                    // [rows][dim] or NULL
    void *out, *y;                      // forward: [rows][dim], each may be NULL
    const void *dout, *dy;              // gradient: [rows][dim], each may be NULL
    void *dx, *dz, *dres;
    float *partial;                     // [blocks][2][dim]: the sums behind dweight and dres_scale, dnext_weight's
    float *dweight, *dres_scale, *dnext_weight;
    long long rows;
    int dim, groups;
    int gate;
    int res_f32;                        // type of res, out, dout, dres (else the I/O type)
    int vec;                            // every row starts on a 16-byte boundary
    float eps;
    // rows brought through a ring of shared-memory stages (set by the launcher): bytes
    // of a stage, where z, res, dy and dout stand in it
    int stages, stage_bytes, off_z, off_res, off_dy, off_dout;
    int *status;                        // the library's device error word
};
cudaError_t launch_block_norm_fwd(const BlockNormParams &p, bool bf16, cudaStream_t stream);
cudaError_t launch_block_norm_bwd(const BlockNormParams &p, bool bf16, cudaStream_t stream);
// Sizes `partial`.
int block_norm_bwd_blocks(long long rows, int dim);

}  // namespace selscan
