// libfa.so, compiled as one unit: the attention calls, then the serving operators, which share the first's device
// state (one status word per device) and argument checks.
#include "fa_api.cu"

#include "serving_api.cuh"
