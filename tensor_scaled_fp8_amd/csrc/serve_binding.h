// The serving operators' part of the compiled binding.
#pragma once

#include <torch/extension.h>

// adds them to the module; library: the handle of the libfp8lin that is loaded
void bind_serve(pybind11::module_& m, void* library);
