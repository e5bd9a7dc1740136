// The whole library as one translation unit, so that all kernels share the device status word
// without relocatable device code.
#include "drscan.cu"

#include "layer.cu"
