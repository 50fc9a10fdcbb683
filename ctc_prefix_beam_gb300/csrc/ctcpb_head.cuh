// Shared by the label head's kernels (layer norm, log-probabilities, cross
// entropy): limits and includes.
#pragma once

#include "ctcpb_kernels.h"
#include "ctcpb_mma.cuh"

namespace ctcpb {

typedef unsigned short u16;

constexpr long long kHeadMaxRows = 1 << 24;  // rows (frames) of a call
constexpr int kHeadMaxWidth = 8192;         // features of a row

}  // namespace ctcpb
