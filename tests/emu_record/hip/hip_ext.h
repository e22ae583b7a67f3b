// Test infrastructure: see ../../emu/hip/hip_ext.h
#pragma once
#include <hip/hip_runtime.h>
#define hipExtLaunchKernelGGL(K, G, B, SH, ST, E0, E1, FL, ...) emu_record(#K, G, B, __VA_ARGS__)
